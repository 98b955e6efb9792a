"""Load-to-LDS reads its LDS address from M0, and the hardware wants a wait state between a
write of M0 and such a load.  The compiler keeps it for its own loads; dma16 is written as
assembly, so its generated code is looked at here."""
import os
import re
import shutil
import subprocess

import pytest

from vocab_wide_add_amd import build

SOURCE = """
#include "device_common.h"
__global__ void copy(const uint16_t* src, uint32_t* dst, uint32_t to)
{
    __shared__ __align__(16) uint32_t s[4096];
    xpress::dma16<%s>(src + threadIdx.x * 8, to);
    xpress::dma16<%s>(src + 4096 + threadIdx.x * 8, to + 1024);
    xpress::wait_vmcnt<0>();
    __syncthreads();
    dst[threadIdx.x] = s[threadIdx.x];
}
"""


@pytest.mark.skipif(not (os.path.exists(build.HIPCC) or shutil.which(build.HIPCC)), reason="needs the compiler")
@pytest.mark.parametrize("once", ["false", "true"])
def test_an_instruction_stands_between_m0_and_the_load(tmp_path, once):
    src, out = tmp_path / "copy.hip", tmp_path / "copy.s"
    src.write_text(SOURCE % (once, once))
    subprocess.run([build.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-S", "--cuda-device-only",
                    "-I", os.path.join(build.PKG, "csrc"), "-o", str(out), str(src)], check=True,
                   capture_output=True, timeout=300)
    code = [x.split(";")[0].strip() for x in out.read_text().splitlines()]
    code = [x for x in code if x and not x.startswith(".") and not x.endswith(":")]
    loads = [i for i, x in enumerate(code) if x.startswith("global_load_lds")]
    assert len(loads) == 2
    for i in loads:
        assert not re.match(r"s_\w+ m0,", code[i - 1]), code[i - 4:i + 1]
