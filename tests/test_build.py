"""What the build refuses (hipcc, no GPU)."""
import subprocess

import pytest

from gated_deltanet_chunked_delta_amd import build


@pytest.mark.parametrize("asm,fine", [
    ('asm volatile("s_mov_b32 m0, %0" :: "s"(n) : "m0")', False),        # written behind the compiler's back
    ('asm volatile("s_nop 0" :: "{m0}"(n))', True)])
def test_assembly_that_writes_a_reserved_register_is_refused(tmp_path, asm, fine):
    src = tmp_path / "k.hip"
    src.write_text("#include <hip/hip_runtime.h>\n__global__ void k(int n) { %s; }\n" % asm)
    r = subprocess.run(["hipcc", "-c", *build.FLAGS, str(src), "-o", str(tmp_path / "k.o")], capture_output=True, text=True)
    assert (r.returncode == 0) == fine, r.stderr
    assert fine or "reserved register" in r.stderr
