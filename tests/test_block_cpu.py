"""Host-side tests of the layer's operators that need no GPU: the library
exports every function include/block.h declares, the binding's structures and
constants match it, and the prepare calls reject every malformed configuration
before touching the HIP runtime."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

from latent_projection_top_amd import block, route

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "block.h")


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_function():
    declared = set(re.findall(r"\b(block_[a-z0-9_]+)\s*\(", header()))
    assert declared == set(block.SYMBOLS)
    lib = ctypes.CDLL(route.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name


def test_binding_matches_header():
    src = header()
    d = {k: int(v) for k, v in re.findall(r"#define\s+(BLOCK_\w+)\s+(\d+)u?", src)}
    assert d["BLOCK_ABI_VERSION"] == block.ABI_VERSION
    assert (d["BLOCK_MAX_ROWS"], d["BLOCK_MAX_SIZE"], d["BLOCK_MAX_STRIDE"]) == (
        block.MAX_ROWS, block.MAX_SIZE, block.MAX_STRIDE)
    enums = {k: int(v) for k, v in re.findall(r"\b(BLOCK_[A-Z0-9_]+)\s*=\s*(\d+)", src)}
    assert [enums[k] for k in ("BLOCK_BF16", "BLOCK_F16", "BLOCK_F32")] == list(block.DTYPES.values())
    for name, code in block.ACTIVATIONS.items():
        assert enums["BLOCK_ACT_" + name.upper()] == code
    for struct, cls in (("block_norm_config", block.NormConfig), ("block_gated_config", block.GatedConfig),
                        ("block_linear_config", block.LinearConfig)):
        body = re.search(r"typedef struct \{([^}]*)\} " + struct, src).group(1)
        fields = re.findall(r"(uint32_t|int32_t|float)\s+(\w+);", body)
        ctype = {"uint32_t": ctypes.c_uint32, "int32_t": ctypes.c_int32, "float": ctypes.c_float}
        assert [(n, ctype[t]) for t, n in fields] == list(cls._fields_)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text("#include \"block.h\"\nint main(void) { block_norm_plan* p;\n"
                   "return block_norm_prepare(0, &p) == ROUTE_E_ARG && block_gated_workspace_bytes(0) == 0 ? 0 : 1; }\n")
    exe = tmp_path / "use"
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), route.LIB_PATH,
                        f"-Wl,-rpath,{os.path.dirname(route.LIB_PATH)}", "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


NORM = dict(abi_version=1, device=0, rows=4, width=8, dtype=0, param_dtype=2, eps=1e-5)
GATED = dict(abi_version=1, device=0, rows=4, inputs=8, inner=8, dtype=0, activation=2, training=0)
LINEAR = dict(abi_version=1, device=0, rows=4, inputs=8, outputs=8, dtype=0, activation=0, training=0)
CONFIG = {"norm": (block.NormConfig, NORM), "gated": (block.GatedConfig, GATED),
          "linear": (block.LinearConfig, LINEAR)}
REFUSED = (
    [("norm", k, v, route.E_ARG) for k, v in (("abi_version", 0), ("abi_version", 2), ("dtype", -1), ("dtype", 3),
                                              ("param_dtype", 3), ("eps", 0.0), ("eps", -1.0),
                                              ("eps", math.inf), ("eps", math.nan))]
    + [("norm", "width", v, route.E_SHAPE) for v in (0, -1, block.MAX_SIZE + 1)]
    + [("norm", "rows", v, route.E_ROWS) for v in (0, -5, block.MAX_ROWS + 1)]
    + [("norm", "device", -1, route.E_DEVICE)])
for _op, _n in (("gated", "inner"), ("linear", "outputs")):
    REFUSED += [(_op, k, v, route.E_ARG) for k, v in (("abi_version", 9), ("dtype", 2), ("dtype", -1),
                                                      ("activation", -1), ("activation", 5))]
    REFUSED += [(_op, k, v, route.E_SHAPE) for k in ("inputs", _n) for v in (0, -1, block.MAX_SIZE + 1)]
    REFUSED += [(_op, "rows", v, route.E_ROWS) for v in (0, -1, block.MAX_ROWS + 1)]
    REFUSED += [(_op, "device", -1, route.E_DEVICE)]
REFUSED.append(("gated", "activation", 0, route.E_ARG))


@pytest.mark.parametrize("op,key,value,status", REFUSED)
def test_prepare_refuses(op, key, value, status):
    cls, base = CONFIG[op]
    assert block.prepare_raw(op, cls(**{**base, key: value})) == (status, 0)


@pytest.mark.parametrize("op", CONFIG)
def test_prepare_order_of_checks(op):
    """A bad argument is reported before a bad shape, that before bad rows,
    and all of them before the device is looked for."""
    cls, base = CONFIG[op]
    size = "width" if op == "norm" else "inputs"
    bad = {"dtype": 7, size: 0, "rows": 0, "device": 4096}
    for key, status in (("dtype", route.E_ARG), (size, route.E_SHAPE), ("rows", route.E_ROWS),
                        ("device", route.E_DEVICE)):
        assert block.prepare_raw(op, cls(**{**base, **bad}))[0] == status
        del bad[key]


@pytest.mark.parametrize("op", CONFIG)
def test_null_arguments(op):
    assert block.prepare_raw(op, None) == (route.E_ARG, 0)
    assert getattr(block.LIB, f"block_{op}_prepare")(None, None) == route.E_ARG
    assert getattr(block.LIB, f"block_{op}_workspace_bytes")(None) == 0
    getattr(block.LIB, f"block_{op}_destroy")(None)
    for call in (f"block_{op}", f"block_{op}_backward"):
        fn = getattr(block.LIB, call)
        assert fn(*[None if t is ctypes.c_void_p else 0 for t in fn.argtypes]) == route.E_ARG


def test_binding_refuses_unknown_names():
    with pytest.raises(ValueError):
        block.NormPlan(4, 8, dtype=torch.float64, device=0)
    with pytest.raises(ValueError):
        block.GatedPlan(4, 8, 8, activation="swish", device=0)
    with pytest.raises(ValueError):
        block.LinearPlan(4, 8, 8, dtype=torch.int8, device=0)
