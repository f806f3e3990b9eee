"""Host-side tests of the routed half of a layer that need no GPU: the library
exports every function include/experts.h declares, the binding's structures and
constants match it, the prepare calls reject every malformed configuration
before touching the HIP runtime, and the 8-bit rounding rule holds."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from latent_projection_top_amd import block, experts, route

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "experts.h")


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_function():
    declared = set(re.findall(r"\b(experts_[a-z0-9_]+)\s*\(", header()))
    assert declared == set(experts.SYMBOLS)
    lib = ctypes.CDLL(route.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name


def test_binding_matches_header():
    src = header()
    d = {k: int(v) for k, v in re.findall(r"#define\s+(EXPERTS_\w+)\s+(\d+)u?", src)}
    assert d["EXPERTS_ABI_VERSION"] == experts.ABI_VERSION
    assert (d["EXPERTS_MAX_COUNT"], d["EXPERTS_MAX_TOPK"], d["EXPERTS_MAX_CHOICES"], d["EXPERTS_MAX_INPUTS"],
            d["EXPERTS_WORKSPACE_ZEROED"]) == (
        experts.MAX_COUNT, experts.MAX_TOPK, experts.MAX_CHOICES, experts.MAX_INPUTS, experts.WORKSPACE_ZEROED)
    for op, cls in (("sort", experts.SortConfig), ("combine", experts.CombineConfig),
                    ("linear8", experts.Linear8Config), ("gated8", experts.Gated8Config)):
        body = re.search(r"typedef struct \{([^}]*)\} experts_" + op + "_config", src).group(1)
        fields = re.findall(r"(uint32_t|int32_t)\s+(\w+);", body)
        ctype = {"uint32_t": ctypes.c_uint32, "int32_t": ctypes.c_int32}
        assert [(n, ctype[t]) for t, n in fields] == list(cls._fields_)


def test_integer_sums_fit_32_bits():
    """|q| <= 127 and |w| <= 128 over the longest reduction."""
    assert 127 * 128 * experts.MAX_INPUTS < 2 ** 31


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text("#include \"experts.h\"\nint main(void) { experts_sort_plan* p;\n"
                   "return experts_sort_prepare(0, &p) == ROUTE_E_ARG && experts_linear8_packed_bytes(0) == 0 ? 0 : 1;"
                   " }\n")
    exe = tmp_path / "use"
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), route.LIB_PATH,
                        f"-Wl,-rpath,{os.path.dirname(route.LIB_PATH)}", "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


SORT = dict(abi_version=1, device=0, rows=4, topk=2, experts=8, first=0)
COMBINE = dict(abi_version=1, device=0, rows=4, topk=2, width=8, dtype=0)
LINEAR8 = dict(abi_version=1, device=0, rows=4, tokens=4, inputs=8, outputs=8, experts=1, dtype=0, activation=0)
GATED8 = dict(abi_version=1, device=0, rows=4, tokens=4, inputs=8, inner=8, experts=1, dtype=0, activation=2)
CONFIG = {"sort": (experts.SortConfig, SORT), "combine": (experts.CombineConfig, COMBINE),
          "linear8": (experts.Linear8Config, LINEAR8), "gated8": (experts.Gated8Config, GATED8)}
REFUSED = []
for _op in CONFIG:
    REFUSED += [(_op, "abi_version", v, route.E_ARG) for v in (0, 2)]
    REFUSED += [(_op, "device", -1, route.E_DEVICE)]
for _op in ("sort", "combine"):
    REFUSED += [(_op, "topk", v, route.E_SHAPE) for v in (0, -1, experts.MAX_TOPK + 1)]
    REFUSED += [(_op, "rows", v, route.E_ROWS) for v in (0, -1, block.MAX_ROWS + 1)]
REFUSED += [("sort", "first", -1, route.E_ARG)]
REFUSED += [("sort", "experts", v, route.E_SHAPE) for v in (0, -1, experts.MAX_COUNT + 1)]
REFUSED += [("combine", "width", v, route.E_SHAPE) for v in (0, block.MAX_SIZE + 1)]
REFUSED += [("combine", "dtype", v, route.E_ARG) for v in (-1, 3)]
for _op, _n in (("linear8", "outputs"), ("gated8", "inner")):
    REFUSED += [(_op, k, v, route.E_ARG) for k, v in (("dtype", 2), ("dtype", -1), ("activation", -1),
                                                      ("activation", 5))]
    REFUSED += [(_op, "inputs", v, route.E_SHAPE) for v in (0, -1, experts.MAX_INPUTS + 1)]
    REFUSED += [(_op, _n, v, route.E_SHAPE) for v in (0, -1, block.MAX_SIZE + 1)]
    REFUSED += [(_op, "experts", v, route.E_SHAPE) for v in (0, experts.MAX_COUNT + 1)]
    REFUSED += [(_op, k, v, route.E_ROWS) for k in ("rows", "tokens") for v in (0, -1, experts.MAX_CHOICES + 1)]
REFUSED.append(("gated8", "activation", 0, route.E_ARG))


@pytest.mark.parametrize("op,key,value,status", REFUSED)
def test_prepare_refuses(op, key, value, status):
    cls, base = CONFIG[op]
    assert experts.prepare_raw(op, cls(**{**base, key: value})) == (status, 0)


@pytest.mark.parametrize("op", ("sort", "combine"))
def test_prepare_refuses_too_many_choices(op):
    cls, base = CONFIG[op]
    assert experts.prepare_raw(op, cls(**{**base, "rows": 1 << 20, "topk": 17})) == (route.E_ROWS, 0)


@pytest.mark.parametrize("op", CONFIG)
def test_prepare_order_of_checks(op):
    cls, base = CONFIG[op]
    size = {"sort": "experts", "combine": "width"}.get(op, "inputs")
    bad = {"abi_version": 7, size: 0, "rows": 0, "device": 4096}
    for key, status in (("abi_version", route.E_ARG), (size, route.E_SHAPE), ("rows", route.E_ROWS),
                        ("device", route.E_DEVICE)):
        assert experts.prepare_raw(op, cls(**{**base, **bad}))[0] == status
        del bad[key]


@pytest.mark.parametrize("op", CONFIG)
def test_null_arguments(op):
    assert experts.prepare_raw(op, None) == (route.E_ARG, 0)
    assert getattr(experts.LIB, f"experts_{op}_prepare")(None, None) == route.E_ARG
    getattr(experts.LIB, f"experts_{op}_destroy")(None)


def test_null_plans():
    for name in experts.SYMBOLS:
        fn = getattr(experts.LIB, name)
        if name.endswith("_bytes"):
            assert fn(None) == 0
        elif not name.endswith(("_prepare", "_destroy")):
            assert fn(*[None if t is ctypes.c_void_p else 0 for t in fn.argtypes]) == route.E_ARG


def test_binding_refuses_unknown_names():
    with pytest.raises(ValueError):
        experts.CombinePlan(4, 2, 8, dtype=torch.float64, device=0)
    with pytest.raises(ValueError):
        experts.Gated8Plan(4, 8, 8, activation="swish", device=0)
    with pytest.raises(ValueError):
        experts.Linear8Plan(4, 8, 8, dtype=torch.int8, device=0)


def rounded(x, a):
    """The device code's quotient, each operation rounded to FP32 (fma once)."""
    f, d = np.float32, np.float64
    up = np.where(a < f(2.0 ** -60), f(2.0 ** 100), np.where(a > f(2.0 ** 60), f(2.0 ** -100), f(1)))
    a = (a * up).astype(f)
    inv = (f(1) / a).astype(f)
    n = (f(127) * (x * up).astype(f)).astype(f)
    t = (n * inv).astype(f)
    # t a has 35 bits and n - t a fewer: exact in FP64, as in the fma
    r = (n.astype(d) - t.astype(d) * a.astype(d)).astype(f)
    # the last fma's exact value needs more than FP64: rounded there first; it
    # decides nothing within 2^-50 of a border but equality, which is kept
    t = (r.astype(d) * inv.astype(d) + t.astype(d)).astype(f)
    return np.rint(t)


@pytest.mark.parametrize("bits", (8, 11))
def test_quantised_integers_are_exact(bits):
    """q = rne(127 x / a) for every significand of x beside random ones of a,
    and every power of two between them that matters, decided in integers."""
    rng = np.random.default_rng(bits)
    half = 1 << (bits - 1)
    mx = np.arange(half, 2 * half)
    for ma in np.unique(np.concatenate((rng.integers(half, 2 * half, 40), [half, 2 * half - 1]))):
        for shift in range(0, 9):
            x = mx[mx <= (ma << shift)]  # x = mx, a = ma 2^shift >= x
            num, den = 127 * x.astype(np.int64), int(ma) << shift
            q, rest = num // den, num % den
            want = q + ((2 * rest > den) | ((2 * rest == den) & (q % 2 == 1)))
            for scale in (0, -120, 80):
                got = rounded(np.ldexp(x.astype(np.float32), scale), np.ldexp(np.float32(den), scale) + 0 * x)
                assert np.array_equal(got.astype(np.int64), want), (ma, shift, scale)
