// bwd_ends.cpp -- test infrastructure, host only.  Runs the main kernel of the causal
// backward (csrc/attn_bwd.cu, unchanged) as one CTA of the model in sm100.cuh beside
// this file.  Nothing of the data is checked; every warp must come to the end, also
// when a copy or a commit is lost or a wait runs out.
//
// usage: bwd_ends d B T G k n_shared sg trials seed mode
// mode: nothing, lost_copy, lost_commit or timeout.  Exit code 1 for a CTA that stays.
#include "sm100.cuh"

namespace gqe {
namespace {
alignas(1024) uint8_t smem_raw[1 << 18];
}
}  // namespace gqe

#include "attn_bwd.cu"

void fake::on_product(uint32_t, uint32_t, bool, uint32_t, bool) {}
void fake::on_tmem_load(uint32_t, int) {}
void fake::on_tmem_store(uint32_t, int) {}
void fake::on_store(uint32_t) {}
void fake::on_copy(uint32_t, const void*, int, int, int, bool) {}
void fake::on_bulk(uint32_t, const void*, uint32_t, bool) {}

int main(int argc, char** argv) {
  using namespace gqe;
  if (argc != 11) return 2;
  int v[9];
  for (int i = 0; i < 9; ++i) v[i] = atoi(argv[i + 1]);
  const std::string mode = argv[10];
  AttnBwdParams p{};
  p.d = v[0], p.B = v[1], p.T = v[2], p.G = v[3], p.k = v[4], p.n_shared = v[5], p.sg = v[6];
  AttnBwdLayout L;
  attn_bwd_layout(p.B, p.T, p.G, p.k, p.n_shared, p.d, &L);
  p.rows_pad = L.rows_pad;
  p.rows_pad_sh = L.rows_pad_sh;
  p.n_rows_pad = L.n_rows_pad;
  std::vector<gqe_bf16_t> dK((size_t)p.B * p.G * p.T * p.d), dV(dK.size());
  p.dK = dK.data();
  p.dV = dV.data();
  CUtensorMap m{};
  fake::base = smem_raw;
  int gave_up = 0;
  for (int t = 0; t < v[7]; ++t) {
    fake::rng.seed(v[8] + t);
    for (double& w : fake::weight) w = 1.0;
    fake::weight[fake::kProduct] = 4.0;
    blockIdx.x = fake::rng() % (unsigned)((p.T + 127) / 128 * p.B * p.G);
    fake::lose_kind = mode == "lost_copy" ? fake::kCopy : fake::kCommit;
    fake::lose = mode == "lost_copy" || mode == "lost_commit" ? (int)(fake::rng() % 60u) : -1;
    fake::timeout_at = mode == "timeout" ? (long)(fake::rng() % 6000u) : -1;
    const bool ok = fake::run_cta(16, [&] {
      p.d == 64 ? attn_bwd_kernel<64>(m, m, m, m, m, m, m, p) : attn_bwd_kernel<128>(m, m, m, m, m, m, m, p);
    });
    gave_up += fake::aborted;
    if (!ok || (mode == "nothing" && fake::aborted)) {
      printf("trial %d: %s\n", t, ok ? "a wait ran out" : fake::error.c_str());
      return 1;
    }
  }
  printf("%d trials, %d gave up\n", v[7], gave_up);
  return 0;
}
