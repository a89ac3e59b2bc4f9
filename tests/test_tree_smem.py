"""The shared memory of the attention kernels over a paged cache: what their code reaches in
each area lies before the next area and within what the launch asks for.  The layouts are
compiled from the kernels' own header, and nothing runs on a GPU."""

import os
import shutil
import subprocess

import pytest

from context_causal_attention_cp_gb300 import build

# The bytes that the kernels' code reaches in each area, counted from that code.
PROBE = r"""
#include <cstdio>
#include "attn_tree_smem.cuh"
using namespace cpattn;

static void area(const char* name, long long at, long long bytes) {
  if (bytes > 0) std::printf("%s %lld %lld\n", name, at, bytes);
}
template <int D, bool QUANT, bool DUAL>
static void mma(const char* name) {
  using C = MmaCfg<D, QUANT, DUAL>;
  std::printf("kernel %s %d 1\n", name, C::kSmemBytes);
  area("queries", 0, 2LL * BM * D * 2);
  area("ring", C::kRingOff, (long long)C::kStages * BN * D * 2);
  area("codes", C::kRawOff, (long long)C::kRawStages * BN * D);
  area("scales", C::kScaleOff, C::kRawStages * BN * 2LL * sizeof(float));
  area("notes", C::kNoteOff, C::kRawStages * (long long)sizeof(RawNote));
  area("tile_exponents", C::kExpOff, 8 * sizeof(int2));
  // (the exponents of every piece that may lie in the ring)
  static_assert(C::kLifts == sizeof(Pieces::at) / sizeof(TreePiece), "places of the piece ring");
  area("query_exponents", C::kLiftOff, QUANT ? (long long)C::kLifts * (DUAL ? 2 : 1) * BM : 0);
  area("scales_of_new_keys", C::kTailOff, C::kTails * 2LL * BN * sizeof(float));
  area("sums_of_streams", C::kMlOff, DUAL ? 0 : 2 * BM * (long long)sizeof(float2));
  area("output_exponents", C::kEvOff, QUANT && !DUAL ? 2 * BM : 0);
  area("bad_rows", C::kBadOff, 16 * 4 + (QUANT ? C::kStages * 4 * 4 : 0));
  area("pieces", C::kPiecesOff, sizeof(Pieces));
  area("barriers", C::kBarOff, (2 * C::kStages + 2 * C::kRawStages + 5 * 2 + 1) * 8);
  area("words", C::kWordOff, 4 * 4 + 2 * 8);  // TMEM, abort, issued[2]; found[2]
  area("sums_of_warps", C::kSumOff, C::kThreads / 32 * 8);
}
template <int D, bool QUANT, int NQ>
static void small(const char* name) {
  using C = TreeCfg<D, QUANT, NQ>;
  std::printf("kernel %s %d 1024\n", name, C::kSmemBytes - 1024);  // (behind its alignment)
  area("tiles", 0, (long long)C::kStages * BN * D * (QUANT ? 1 : 2));
  area("scales", C::kScaleOff, QUANT ? C::kStages * BN * 4 : 0);
  area("queries", C::kQOff, 2LL * 8 * NQ * D * 2);
  area("join", C::kJoinOff, 8LL * 8 * NQ * D * 4);
  area("sums_of_warps", C::kMlOff, 8LL * 8 * NQ * 8);
  area("pieces", C::kPiecesOff, sizeof(Pieces));
  area("barriers", C::kBarOff, (2 * C::kStages + 4) * 8);
  area("words", C::kWordOff, 16 + 2 * 8);  // abort, issued[2]; found[2]
  area("sums", C::kSumOff, kSmallThreads / 32 * 8);
}
int main() {
  mma<128, true, true>("mma_128_e4m3_dual");
  mma<128, true, false>("mma_128_e4m3_single");
  mma<64, true, true>("mma_64_e4m3_dual");
  mma<64, true, false>("mma_64_e4m3_single");
  mma<128, false, true>("mma_128_bf16_dual");
  mma<128, false, false>("mma_128_bf16_single");
  mma<64, false, true>("mma_64_bf16_dual");
  mma<64, false, false>("mma_64_bf16_single");
  small<128, true, 1>("small_128_e4m3_8");
  small<128, true, 2>("small_128_e4m3_16");
  small<64, true, 1>("small_64_e4m3_8");
  small<64, true, 2>("small_64_e4m3_16");
  small<128, false, 1>("small_128_bf16_8");
  small<128, false, 2>("small_128_bf16_16");
  small<64, false, 1>("small_64_bf16_8");
  small<64, false, 2>("small_64_bf16_16");
  return 0;
}
"""
KERNELS = [f"mma_{d}_{k}_{u}" for d in (64, 128) for k in ("bf16", "e4m3") for u in ("single", "dual")] + \
    [f"small_{d}_{k}_{r}" for d in (64, 128) for k in ("bf16", "e4m3") for r in (8, 16)]


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no nvcc")
    at = tmp_path_factory.mktemp("layouts")
    (at / "probe.cu").write_text(PROBE)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC,
                    str(at / "probe.cu"), "-o", str(at / "probe")], check=True, capture_output=True)
    out = subprocess.run([str(at / "probe")], check=True, capture_output=True, text=True).stdout
    kernels = {}
    for line in out.splitlines():
        w = line.split()
        if w[0] == "kernel":
            areas = kernels[w[1]] = [("end", int(w[2]), 0)]
        else:
            areas.insert(-1, (w[0], int(w[1]), int(w[2])))
    return kernels


@pytest.mark.parametrize("name", KERNELS)
def test_areas_hold_what_the_code_reaches(name, layouts):
    areas = layouts[name]
    assert areas[-1][1] <= 227 * 1024
    for (what, at, size), (_, after, _) in zip(areas, areas[1:]):
        assert at >= 0 and at + size <= after, f"{what}: {at} + {size} reach past {after}"
