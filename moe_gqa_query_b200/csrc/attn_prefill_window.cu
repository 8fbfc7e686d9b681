// attn_prefill_window.cu -- routed causal attention under a sliding window with
// sinks, for the prefill, on tcgen05.
//
// The rows are attn_prefill.cu's: the (t, j) rows of a group packed into 128-row
// query tiles, and the shared head's rows against group sg.  Query t sees key p
// when p <= t and (p > t - window or p < sinks), so a query tile walks a list of
// key tiles instead of the prefix: the tiles that hold sinks, and the tiles from
// its first row's window start to its last row.  Masks are applied on the tiles
// that hold a border of the visible set.  A row may see nothing of a tile (its
// window starts behind it): its running max stays -inf, its exponentials are
// taken against 0 and come out 0.
//
// One query tile per CTA of 192 threads in 256 tensor-memory columns, two CTAs
// per SM, at both head widths: key tiles of 128 keys at d = 64 (S 0 | P 128 |
// O 192) and of 64 keys at d = 128 (S 0 | P 64 | O 128), so that S, P and O have
// columns of their own and S(j+1) runs while the exponentials of tile j do.  The
// walks are short (window / 128 + 2 tiles), so a CTA's start and end count, and
// two independent CTAs hide each other's.
//
// With at most 32 sinks the sink tile is narrow: 32 of its keys take part in
// S, the softmax and P V.
//
// Warp 4 brings K by TMA and issues S = Q K^T, warp 5 brings V and issues
// O += P V, warps 0-3 do the softmax, one row per thread: S once into registers,
// row max in the base-2 domain, O rescaled only when the max grows by more than
// 2^8, P (bf16) to tensor memory.  At d = 64 P is announced in two halves
// (p_half, p_full), so its first half's products overlap the second half's
// exponentials; one thread issues them all in order, so the result does not
// depend on timing.
#include "attn.cuh"
#include "launch.cuh"

namespace gqe {

namespace {

constexpr int kRowsPW = 128;          // query rows per tile
constexpr int kThreadsPW = 192;
constexpr int kNarrow = 32;           // keys of a narrow sink tile
constexpr float kRescalePW = 8.0f;
// Column pairs of every 16 whose exponentials run as the FMA-pipe polynomial at
// d = 64, as in attn_prefill.cu's short walks.
constexpr int kPolyPW = 2;

struct __align__(8) PrefillWinBarriers {
  uint64_t q_full;
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full, s_free, p_half, p_full, pv_done;
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct PrefillWinCfg {
  static constexpr int NB = D / 64;
  static constexpr int KT = D == 64 ? 128 : 64;
  static constexpr bool kHalves = KT == 128;
  static constexpr int KST = D == 64 ? 3 : 2, VST = 2;       // ring depths
  static constexpr int QBox = kRowsPW * 128, KBox = KT * 128; // 64 columns wide
  static constexpr int QBytes = NB * QBox, KVBytes = NB * KBox;
  static constexpr uint32_t kS = 0, kP = KT, kO = D == 64 ? 192 : 128;
  static constexpr size_t Smem = 1024 + QBytes + (KST + VST) * KVBytes + sizeof(PrefillWinBarriers);
};

// The key tiles a query tile walks: 0 .. n_sink-1, then w0, w0+1, ...
struct KeyList {
  int n, n_sink, w0;
  __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : w0 + j - n_sink; }
};

struct RowTile {
  float m, l;       // running max (base 2) and sum of the row
  bool ok;
};

// One tile: NC of its keys (from its first), base the position of the first.
template <int D, int NC>
__device__ __forceinline__ void softmax_tile(RowTile& st, PrefillWinBarriers* bar, uint32_t lane_base, int j, int base,
                                             int t_r, bool diag, bool border, const AttnParams& p,
                                             volatile int* abort) {
  using C = PrefillWinCfg<D>;
  constexpr int NH = C::kHalves && NC == 128 ? 2 : 1;      // P in halves
  const float sl2 = p.scale_log2;
  uint32_t s[NC];
  tmem_ld<NC>(lane_base + C::kS, s);
  tc_fence_before();
  mbar_arrive(&bar->s_free);       // S(j) is in registers
  if (diag || border) {
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += 32) {
      const int pos = base + c0;
      const uint32_t vis =
          bits_below(t_r + 1, pos) & (~bits_below(t_r - p.window + 1, pos) | bits_below(p.sinks, pos));
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!((vis >> c) & 1u)) s[c0 + c] = __float_as_uint(-INFINITY);
    }
  }
  float m8[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) m8[q] = -INFINITY;
#pragma unroll
  for (int c = 0; c < NC / 2; ++c)
    m8[c & 7] = fmax3(m8[c & 7], __uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
  const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                         fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
  const float m_new = fmaxf(st.m, mx * sl2);
  bool rescale = false;
  float alpha = 1.f;
  if (j == 0) {
    st.m = m_new;
  } else {
    const bool need = m_new > st.m + kRescalePW;
    rescale = __any_sync(0xffffffffu, need);
    if (need) {
      alpha = ex2(st.m - m_new);
      st.l *= alpha;
      st.m = m_new;
    }
  }
  const float neg_m = st.m == -INFINITY ? 0.f : -st.m;       // nothing seen yet: every exponential is 0
  const unsigned long long sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg_m, neg_m);
  unsigned long long sum2[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    constexpr int PC = NC / 2 / NH;        // pairs of this half
    uint32_t pk[PC];
#pragma unroll
    for (int c = 0; c < PC; ++c) {
      const int q = h * PC + c;
      const unsigned long long x =
          f2_fma(f2_pack(__uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1])), sl2x2, negm2);
      float p0, p1;
      if (D == 64 && (c & 15) < kPolyPW) {
        exp2_poly2(x, p0, p1);
      } else {
        float x0, x1;
        f2_unpack(x, x0, x1);
        p0 = ex2(x0);
        p1 = ex2(x1);
      }
      sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(p0, p1));
      pk[c] = pack_bf16x2(p0, p1);
    }
    if (h == 0 && j > 0) {
      // P(j-1) V must be done before P is overwritten and O rescaled
      st.ok = mbar_wait_short(&bar->pv_done, (j - 1) & 1, abort) && st.ok;
      tc_fence_after();
      if (rescale) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(lane_base + C::kO + c0, o);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tmem_st32(lane_base + C::kO + c0, o);
        }
      }
    }
    tmem_st<PC>(lane_base + C::kP + h * PC, pk);
    tmem_wait_st();
    tc_fence_before();
    if (C::kHalves && h == 0) mbar_arrive(&bar->p_half);
    if (h == NH - 1) mbar_arrive(&bar->p_full);
  }
  float a0, a1, b0, b1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  st.l += (a0 + a1) + (b0 + b1);
}

template <int D>
__global__ void __launch_bounds__(kThreadsPW, 2)
attn_prefill_window_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapQs,
                           const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                           AttnParams p) {
  using C = PrefillWinCfg<D>;
  constexpr int KT = C::KT, KST = C::KST, VST = C::VST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::QBytes;
  uint8_t* sV = sK + KST * C::KVBytes;
  PrefillWinBarriers* bar = reinterpret_cast<PrefillWinBarriers*>(sV + VST * C::KVBytes);
  volatile int* abort = &bar->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item: one query tile, from the sequence's end on (full walks first)
  const int BG = p.B * p.G;
  const int per_level = BG * p.k + p.B * p.n_shared;
  const int n_levels = (p.T + kRowsPW - 1) / kRowsPW;
  const int level = n_levels - 1 - (int)blockIdx.x / per_level;
  const int i = blockIdx.x % per_level;
  const bool routed = i < BG * p.k;
  const int seq = routed ? i % BG : i - BG * p.k;
  const int row0 = (routed ? level * p.k + i / BG : level) * kRowsPW;
  const int kvseq = routed ? seq : seq * p.G + p.sg;
  const int kk = routed ? p.k : 1;
  const int rows_total = p.T * kk;
  if (row0 >= rows_total) return;
  const int t_first = row0 / kk, t_last = min(p.T - 1, (row0 + kRowsPW - 1) / kk);
  KeyList kl;
  kl.w0 = max(0, t_first - p.window + 1) / KT;
  kl.n_sink = min((p.sinks + KT - 1) / KT, kl.w0);
  kl.n = kl.n_sink + t_last / KT + 1 - kl.w0;
  // the first entry is a sink tile of which at most kNarrow keys count
  const bool narrow = kl.n_sink == 1 && p.sinks <= kNarrow;
  const CUtensorMap* mq = routed ? &mapQ : &mapQs;

  auto load_k = [&](int j) {
    const int s = j % KST;
    mbar_arrive_expect_tx(&bar->k_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sK + s * C::KVBytes + bx * C::KBox, &mapK, &bar->k_full[s], bx * 64, kl.tile(j) * KT, kvseq);
  };
  auto load_v = [&](int j) {
    const int s = j % VST;
    mbar_arrive_expect_tx(&bar->v_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sV + s * C::KVBytes + bx * C::KBox, &mapV, &bar->v_full[s], bx * 64, kl.tile(j) * KT, kvseq);
  };
  // the barriers, Q and the first K and V tiles before the CTA-wide barrier, so
  // that they load while tensor memory is allocated
  if (warp == 4 && lane == 0) {
    mbar_init(&bar->q_full, 1);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
    }
    mbar_init(&bar->s_full, 1);
    mbar_init(&bar->s_free, 128);
    mbar_init(&bar->p_half, 128);
    mbar_init(&bar->p_full, 128);
    mbar_init(&bar->pv_done, 1);
    bar->abort = 0;
    fence_mbar_init();
    pdl_wait();
    mbar_arrive_expect_tx(&bar->q_full, C::QBytes);
    for (int bx = 0; bx < C::NB; ++bx) tma_load_3d(sQ + bx * C::QBox, mq, &bar->q_full, bx * 64, row0, seq);
    for (int j = 0; j < KST && j < kl.n; ++j) {
      load_k(j);
      if (j < VST) load_v(j);
    }
  }
  __syncwarp();
  if (warp == 5) tmem_alloc(&bar->tmem_base, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 4) {
    // ---------------- K side: S(j+1) is issued as soon as the softmax holds S(j)
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_bf16_f32(kRowsPW, KT, false, false);
    constexpr uint32_t idesc_n = idesc_bf16_f32(kRowsPW, kNarrow, false, false);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    bool ok = mbar_wait_warp(&bar->q_full, 0, abort);
    for (int j = 0; ok && j < kl.n; ++j) {
      const int s = j % KST;
      if (j > 0 && !mbar_wait_warp(&bar->s_free, (j - 1) & 1, abort)) break;
      if (!mbar_wait_warp(&bar->k_full[s], (j / KST) & 1, abort)) break;
      tc_fence_after();
      if (leader) {
        const uint64_t dk = sdesc_sw128(smem_u32(sK + s * C::KVBytes), 16, 1024);
        const uint32_t idesc = narrow && j == 0 ? idesc_n : idesc_s;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_ss(tmem + C::kS, sdesc_at(dq, (ks >> 2) * C::QBox + (ks & 3) * 32),
                  sdesc_at(dk, (ks >> 2) * C::KBox + (ks & 3) * 32), idesc, ks > 0);
        umma_commit(&bar->s_full);
        umma_commit(&bar->k_empty[s]);
      }
      if (j + KST < kl.n) {
        if (!mbar_wait_warp(&bar->k_empty[s], (j / KST) & 1, abort)) break;
        if (leader) load_k(j + KST);
      }
    }
  } else if (warp == 5) {
    // ---------------- V side: O += P(j) V_j
    const bool leader = elect_one();
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRowsPW, D, false, true);
    for (int j = 0; j < kl.n; ++j) {
      const int s = j % VST;
      const bool half = C::kHalves && !(narrow && j == 0);
      const int steps = narrow && j == 0 ? kNarrow / 16 : KT / 16;
      if (!mbar_wait_warp(C::kHalves ? &bar->p_half : &bar->p_full, j & 1, abort)) break;
      if (!mbar_wait_warp(&bar->v_full[s], (j / VST) & 1, abort)) break;
      tc_fence_after();
      const uint64_t dv = sdesc_sw128(smem_u32(sV + s * C::KVBytes), C::KBox, 1024);
      const int first = half ? steps / 2 : steps;
      if (leader)
#pragma unroll 4
        for (int ks = 0; ks < first; ++ks)
          umma_ts(tmem + C::kO, tmem + C::kP + ks * 8, sdesc_at(dv, ks * 2048), idesc_o, (j > 0 || ks > 0));
      if (C::kHalves) {
        if (!mbar_wait_warp(&bar->p_full, j & 1, abort)) break;
        tc_fence_after();
        if (leader)
#pragma unroll 4
          for (int ks = first; ks < steps; ++ks)
            umma_ts(tmem + C::kO, tmem + C::kP + ks * 8, sdesc_at(dv, ks * 2048), idesc_o, 1u);
      }
      if (leader) {
        umma_commit(&bar->pv_done);
        umma_commit(&bar->v_empty[s]);
      }
      if (j + VST < kl.n) {
        if (!mbar_wait_warp(&bar->v_empty[s], (j / VST) & 1, abort)) break;
        if (leader) load_v(j + VST);
      }
    }
  } else {
    // ---------------- softmax: warps 0-3, one query row per thread
    const int prow = row0 + warp * 32 + lane;
    const int t_r = prow / kk;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    RowTile st{-INFINITY, 0.f, true};
    for (int j = 0; j < kl.n && st.ok; ++j) {
      const int base = kl.tile(j) * KT;
      const bool diag = base + KT - 1 > t_first;
      const bool border = base < t_last - p.window + 1 && base + KT > p.sinks;
      st.ok = mbar_wait_short(&bar->s_full, j & 1, abort);
      tc_fence_after();
      if (narrow && j == 0)
        softmax_tile<D, kNarrow>(st, bar, lane_base, j, base, t_r, diag, true, p, abort);
      else
        softmax_tile<D, KT>(st, bar, lane_base, j, base, t_r, diag, border, p, abort);
    }
    // ---------------- epilogue: O / l -> bf16
    st.ok = mbar_wait_short(&bar->pv_done, (kl.n - 1) & 1, abort) && st.ok;
    tc_fence_after();
    const bool valid = prow < rows_total && st.ok;
    const float inv_l = 1.f / st.l;
    gqe_bf16_t* orow = (routed ? p.o_routed : p.o_sh) + ((size_t)seq * rows_total + prow) * D;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 64) {
      uint32_t o[64];
      tmem_ld64(lane_base + C::kO + c0, o);
      if (valid) {
        uint4* d4 = reinterpret_cast<uint4*>(orow + c0);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pk[e] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * e]) * inv_l, __uint_as_float(o[8 * c + 2 * e + 1]) * inv_l);
          d4[c] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
    }
    if (p.lse && valid)
      p.lse[(routed ? 0 : (size_t)BG * p.T * p.k) + (size_t)seq * rows_total + prow] =
          (st.m + __log2f(st.l)) * 0.69314718055994531f;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  report_abort(abort, p.err, kErrTimeoutAttn);
  drain_after_abort(abort);
}

}  // namespace

template <int D>
static cudaError_t launch_win(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mK,
                              const CUtensorMap& mV, const AttnParams& p, cudaStream_t stream) {
  const size_t smem = PrefillWinCfg<D>::Smem;
  auto kern = attn_prefill_window_kernel<D>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int n_levels = (p.T + kRowsPW - 1) / kRowsPW;
  const int per_level = p.B * p.G * p.k + p.B * p.n_shared;
  return launch_kernel(kern, dim3(n_levels * per_level), dim3(kThreadsPW), smem, stream, 1, mQ, mQs, mK, mV, p);
}

cudaError_t launch_attn_prefill_window(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mK,
                                       const CUtensorMap& mV, const AttnParams& p, int d, cudaStream_t stream) {
  return d == 64 ? launch_win<64>(mQ, mQs, mK, mV, p, stream) : launch_win<128>(mQ, mQs, mK, mV, p, stream);
}

}  // namespace gqe
