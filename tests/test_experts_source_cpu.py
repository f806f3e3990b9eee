"""What the routed half's kernels rest on, read in their sources: the built
kernels may have it right by chance."""
import os
import re
import shutil
import subprocess

import pytest

from latent_projection_top_amd import build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "latent_projection_top_amd", "csrc")


def kernels(name):
    """{kernel: body without comments} of a source."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    out = {}
    for m in re.finditer(r"\bvoid (\w+_kernel)\([^{;]*\)\s*\{", src):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        out[m.group(1)] = src[m.end():end]
    return out


def test_lanes_that_hold_choices_stay_until_they_are_read():
    """Places and weights are read out of the lanes that hold them, one choice
    to a lane whatever the row's width: no lane may leave between the two."""
    bodies = kernels("experts_rows.hip")
    assert {"gather_kernel", "collect_kernel", "backward_kernel"} <= set(bodies)
    for name, body in bodies.items():
        if "Choices k(" not in body:
            continue
        held = body[body.index("Choices k("):]
        reads = [m.end() for m in re.finditer(r"k\.next\(|readlane\(", held)]
        assert reads, name
        assert not re.search(r"\breturn\b", held[:reads[-1]]), name


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="no hipcc")
@pytest.mark.parametrize("name", ["experts_rows.hip", "experts_sort.hip", "experts_quantise.hip"])
def test_no_arithmetic_in_doubles(name, tmp_path):
    """Counts are integers and sums FP32: an FP64 instruction is a call that
    resolved to another overload than was meant."""
    out = str(tmp_path / "kernels.s")
    r = subprocess.run([build.HIPCC, *build.COMMON_FLAGS, *build.EXTRA_FLAGS.get(name, []), "--cuda-device-only", "-S",
                        os.path.join(CSRC, name), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    doubles = set(re.findall(r"\bv_\w+_f64\w*", open(out).read()))
    assert not doubles, doubles


def test_bare_barriers_stand_between_fences():
    """A barrier that orders no memory by itself: what was stored before it is
    released, what is read after it acquired, in the source and not only in the
    order that the compiler chose."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.startswith("experts"):
            continue
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__builtin_amdgcn_s_barrier\(\);", src):
            found += 1
            before, after = src[:m.start()].rstrip(), src[m.end():].lstrip()
            assert re.search(r"__builtin_amdgcn_fence\(__ATOMIC_RELEASE, \"workgroup\"[^;]*\);$", before), name
            assert re.match(r"__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, \"workgroup\"", after), name
    assert found
