"""What the build refuses (hipcc, no GPU)."""
import re
import struct
import subprocess

import pytest

from gated_deltanet_chunked_delta_amd import binding, build

msgpack = pytest.importorskip("msgpack")


@pytest.mark.parametrize("asm,fine", [
    ('asm volatile("s_mov_b32 m0, %0" :: "s"(n) : "m0")', False),        # written behind the compiler's back
    ('asm volatile("s_nop 0" :: "{m0}"(n))', True)])
def test_assembly_that_writes_a_reserved_register_is_refused(tmp_path, asm, fine):
    src = tmp_path / "k.hip"
    src.write_text("#include <hip/hip_runtime.h>\n__global__ void k(int n) { %s; }\n" % asm)
    r = subprocess.run(["hipcc", "-c", *build.FLAGS, str(src), "-o", str(tmp_path / "k.o")], capture_output=True, text=True)
    assert (r.returncode == 0) == fine, r.stderr
    assert fine or "reserved register" in r.stderr


def kernel_metadata(path):
    """{kernel's name: its entry} of the code objects that a library built here holds."""
    blob, out = open(path, "rb").read(), {}
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := blob.find(magic, at)) >= 0:
        (n,), p = struct.unpack_from("<Q", blob, at + 24), at + 32
        for _ in range(n):
            offset, size, chars = struct.unpack_from("<QQQ", blob, p)
            if b"gfx950" in blob[p + 24:p + 24 + chars]:
                elf = blob[at + offset:at + offset + size]
                shoff, (shentsize, shnum) = struct.unpack_from("<Q", elf, 40)[0], struct.unpack_from("<HH", elf, 58)
                for k in range(shnum):
                    kind, = struct.unpack_from("<I", elf, shoff + k * shentsize + 4)
                    start, length = struct.unpack_from("<QQ", elf, shoff + k * shentsize + 24)
                    if kind != 7:                               # (SHT_NOTE)
                        continue
                    namesz, descsz, _ = struct.unpack_from("<III", elf, start)
                    desc = start + 12 + (namesz + 3) // 4 * 4
                    for entry in msgpack.unpackb(elf[desc:desc + descsz], strict_map_key=False).get("amdhsa.kernels", []):
                        out[entry[".name"]] = entry
            p += 24 + chars
        at += 24
    return out


def test_kernels_keep_their_tiles_in_registers():
    """A loop over accumulators that is not unrolled puts them into memory, at half the speed and without a word."""
    kernels = kernel_metadata(binding.LIB_PATH)
    hot = [n for n in kernels if re.search(r"gemm_kernel|skinny_kernel|rec_(fwd|bwd|step)_kernel|addnorm_(fwd|bwd)_kernel", n)]
    assert len(hot) > 100
    assert {n: kernels[n][".private_segment_fixed_size"] for n in hot if kernels[n][".private_segment_fixed_size"] or kernels[n][".vgpr_spill_count"]} == {}
