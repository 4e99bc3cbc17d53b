"""The forms of gdn_gemm_fp8's kernel on one SM, checked by the compiler (no
GPU needed).

Every form holds tensor memory while its blocks wait for the others of their
cluster, and an allocation waits without a limit. Two kernels on two streams
must therefore never share SMs whose 512 columns are too few for both: each
could hold what a block of the other's cluster waits for."""
import os
import subprocess

from gated_delta_net_02_gb300 import build

CHECK = """
#include "gemm_fp8.cu"
namespace gdn {
namespace {
// 233472 bytes of shared memory an SM, 1024 of them taken for each block
template <class A, class B, int COLS_A, int COLS_B>
constexpr bool apart() {
  return A::SMEM + B::SMEM + 2048 > 233472 || COLS_A + COLS_B <= 512;
}
using S16 = SmallCfg<16, false>;
using S32 = SmallCfg<32, false>;
using S64 = SmallCfg<64, false>;
using Square = SmallCfg<128, true>;
static_assert(S16::TCOLS == 64 && S32::TCOLS == 128 && S64::TCOLS == 256 && Square::TCOLS == 512);
static_assert(apart<S16, S16, 64, 64>() && apart<S16, S32, 64, 128>() &&
              apart<S16, S64, 64, 256>() && apart<S32, S32, 128, 128>() &&
              apart<S32, S64, 128, 256>() && apart<S64, S64, 256, 256>(), "up to 64 rows");
static_assert(apart<Square, S16, 512, 64>(), "square tiles, up to 16 rows");
static_assert(apart<Square, S32, 512, 128>(), "square tiles, up to 32 rows");
static_assert(apart<Square, S64, 512, 256>(), "square tiles, up to 64 rows");
static_assert(apart<Square, Square, 512, 512>(), "square tiles");
static_assert(apart<LargeCfg, S16, 512, 64>() && apart<LargeCfg, S32, 512, 128>() &&
              apart<LargeCfg, S64, 512, 256>() && apart<LargeCfg, Square, 512, 512>() &&
              apart<LargeCfg, LargeCfg, 512, 512>(), "pairs of blocks");
static_assert(3 * (S16::SMEM + 1024) > 233472, "three blocks on an SM");
}  // namespace
}  // namespace gdn
"""


def test_no_two_forms_can_wait_for_each_others_tensor_memory(tmp_path):
    src = tmp_path / "check.cu"
    src.write_text(CHECK)
    r = subprocess.run([build._nvcc()] + build.NVCC_FLAGS + ["-ptx", str(src), "-o", os.devnull],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
