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
// One query tile per CTA of 192 threads, key tiles of 64 keys, S, P and O in
// tensor-memory columns of their own, so that S(j+1) runs while the exponentials
// of tile j do.  The walks are short (window / 64 + 3 tiles), so a CTA's start and
// end count, and one tile's softmax leaves the exponential unit idle between its
// steps; what fills both gaps is independent CTAs on one SM: two at d = 128 (256
// columns: S 0 | P 64 | O 128), three at d = 64 (S 0 | O 64, and 32 columns
// allocated apart for P).  A 32768-token prefill of 9 heads at d = 64 under a
// 1024-token window: two CTAs with 128-key tiles 146 us, four with 64-key tiles
// and P over S, so that S(j+1) waits for P(j) V, 146 us; this form 132 us (133
// and 142 us with 2 and 4 of 16 pairs of exponentials on the FMA-pipe polynomial).
// That is 0.34 of the measured bf16 rate; the exponential unit is 65 % busy, the
// rest are the gaps that are left.  2 x 8192 tokens of 17 heads at d = 128 take 157
// us, 0.52 of it.  (GPU times in a captured graph on one box; others: 131 to 138 us,
// and 157 to 170.)
//
// With at most 32 sinks the sink tile is narrow: 32 of its keys take part in
// S, the softmax and P V.
//
// Warp 4 issues S = Q K^T and O += P V, warp 5 brings Q, K and V by TMA, warps
// 0-3 do the softmax, one row per thread: S once into registers, row max in the
// base-2 domain, O rescaled only when the max grows by more than 2^8, P (bf16)
// to tensor memory.  One thread issues every product in order, so the result
// does not depend on timing.
#include "attn.cuh"
#include "launch.cuh"

namespace gqe {

namespace {

constexpr int kRowsPW = 128;          // query rows per tile
constexpr int kThreadsPW = 192;
constexpr int kNarrow = 32;           // keys of a narrow sink tile
constexpr float kRescalePW = 8.0f;

struct __align__(8) PrefillWinBarriers {
  uint64_t q_full;
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full, s_free, p_full, pv_done;
  uint32_t tmem_base, tmem_p;
  int abort;
};

template <int D>
struct PrefillWinCfg {
  static constexpr int NB = D / 64;
  static constexpr bool kApart = D == 64;                    // P's columns allocated apart
  static constexpr int KT = 64, ST = D == 64 ? 3 : 2;        // keys per tile, K and V ring depth
  static constexpr int QBox = kRowsPW * 128, KBox = KT * 128; // 64 columns wide
  static constexpr int QBytes = NB * QBox, KVBytes = NB * KBox;
  static constexpr uint32_t kS = 0, kO = kApart ? 64 : 128;
  static constexpr uint32_t kCols = kApart ? 128 : 256;
  // CTAs per SM.  At d = 64 shared memory holds three (and not four, whose first
  // blocks of columns would leave none for P)
  static constexpr int kCtas = kApart ? 3 : 2;
  static constexpr size_t Smem = 1024 + QBytes + 2 * ST * KVBytes + sizeof(PrefillWinBarriers);
};

static_assert(4 * (PrefillWinCfg<64>::Smem + 1024) > 228 * 1024, "a fourth CTA would wait for its P columns");

// The key tiles a query tile walks: 0 .. n_sink-1, then w0, w0+1, ...
struct KeyList {
  int n, n_sink, w0;
  __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : w0 + j - n_sink; }
};

struct RowTile {
  float m, l;       // running max (base 2) and sum of the row
  bool ok;
};

// N scores of a row whose token is t_r, from key position pos on: the ones it
// does not see become -inf.
template <int N>
__device__ __forceinline__ void mask_scores(uint32_t* s, int pos, int t_r, const AttnParams& p) {
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += 32) {
    const int q = pos + c0;
    const uint32_t vis = bits_below(t_r + 1, q) & (~bits_below(t_r - p.window + 1, q) | bits_below(p.sinks, q));
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((vis >> c) & 1u)) s[c0 + c] = __float_as_uint(-INFINITY);
  }
}

template <int N>
__device__ __forceinline__ float max_scores(const uint32_t* s) {
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < N / 2; ++c)
    m4[c & 3] = fmax3(m4[c & 3], __uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// One tile: NC of its keys (from its first), base the position of the first.
template <int D, int NC>
__device__ __forceinline__ void softmax_tile(RowTile& st, PrefillWinBarriers* bar, uint32_t lane_base, uint32_t lane_p,
                                             int j, int base, int t_r, bool border, const AttnParams& p,
                                             volatile int* abort) {
  using C = PrefillWinCfg<D>;
  const float sl2 = p.scale_log2;
  uint32_t s[NC];
  tmem_ld<NC>(lane_base + C::kS, s);
  tc_fence_before();
  mbar_arrive(&bar->s_free);       // S(j) is in registers
  if (border) mask_scores<NC>(s, base, t_r, p);
  const float m_new = fmaxf(st.m, max_scores<NC>(s) * sl2);
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
  uint32_t pk[NC / 2];
#pragma unroll
  for (int c = 0; c < NC / 2; ++c) {
    const unsigned long long x =
        f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, negm2);
    float p0, p1;
    f2_unpack(x, p0, p1);
    p0 = ex2(p0);
    p1 = ex2(p1);
    sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(p0, p1));
    pk[c] = pack_bf16x2(p0, p1);
  }
  if (j > 0) {
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
  tmem_st<NC / 2>(lane_p, pk);
  tmem_wait_st();
  tc_fence_before();
  mbar_arrive(&bar->p_full);
  float a0, a1, b0, b1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  st.l += (a0 + a1) + (b0 + b1);
}

template <int D>
__global__ void __launch_bounds__(kThreadsPW, PrefillWinCfg<D>::kCtas)
attn_prefill_window_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapQs,
                           const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                           AttnParams p) {
  using C = PrefillWinCfg<D>;
  constexpr int KT = C::KT, ST = C::ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::QBytes;
  uint8_t* sV = sK + ST * C::KVBytes;
  PrefillWinBarriers* bar = reinterpret_cast<PrefillWinBarriers*>(sV + ST * C::KVBytes);
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
    const int s = j % ST;
    mbar_arrive_expect_tx(&bar->k_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sK + s * C::KVBytes + bx * C::KBox, &mapK, &bar->k_full[s], bx * 64, kl.tile(j) * KT, kvseq);
  };
  auto load_v = [&](int j) {
    const int s = j % ST;
    mbar_arrive_expect_tx(&bar->v_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sV + s * C::KVBytes + bx * C::KBox, &mapV, &bar->v_full[s], bx * 64, kl.tile(j) * KT, kvseq);
  };
  // the barriers, Q and the first K and V tiles before the CTA-wide barrier, so
  // that they load while tensor memory is allocated
  if (warp == 5 && lane == 0) {
    mbar_init(&bar->q_full, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
    }
    mbar_init(&bar->s_full, 1);
    mbar_init(&bar->s_free, 128);
    mbar_init(&bar->p_full, 128);
    mbar_init(&bar->pv_done, 1);
    bar->abort = 0;
    fence_mbar_init();
    pdl_wait();
    mbar_arrive_expect_tx(&bar->q_full, C::QBytes);
    for (int bx = 0; bx < C::NB; ++bx) tma_load_3d(sQ + bx * C::QBox, mq, &bar->q_full, bx * 64, row0, seq);
    for (int j = 0; j < ST && j < kl.n; ++j) {
      load_k(j);
      load_v(j);
    }
  }
  if (warp == 4) {
    if (C::kApart) tmem_alloc2(&bar->tmem_base, C::kCols, &bar->tmem_p, 32);
    else tmem_alloc(&bar->tmem_base, C::kCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base, tmem_p = C::kApart ? bar->tmem_p : tmem + 64;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 4) {
    // ---------------- MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16_f32(kRowsPW, KT, false, false);
    constexpr uint32_t idesc_n = idesc_bf16_f32(kRowsPW, kNarrow, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRowsPW, D, false, true);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    auto issue_s = [&](int j) {
      const int s = j % ST;
      if (!mbar_wait_warp(&bar->k_full[s], (j / ST) & 1, abort)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = sdesc_sw128(smem_u32(sK + s * C::KVBytes), 16, 1024);
        const uint32_t idesc = narrow && j == 0 ? idesc_n : idesc_s;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_ss(tmem + C::kS, sdesc_at(dq, (ks >> 2) * C::QBox + (ks & 3) * 32),
                  sdesc_at(dk, (ks >> 2) * C::KBox + (ks & 3) * 32), idesc, ks > 0);
        umma_commit(&bar->s_full);
        umma_commit(&bar->k_empty[s]);
      }
      return true;
    };
    bool ok = mbar_wait_warp(&bar->q_full, 0, abort);
    for (int j = -1; ok && j < kl.n; ++j) {
      if (j + 1 < kl.n) {
        // S(j+1) as soon as the softmax holds S(j)
        if (j >= 0 && !mbar_wait_warp(&bar->s_free, j & 1, abort)) break;
        if (!issue_s(j + 1)) break;
      }
      if (j >= 0) {
        const int s = j % ST;
        if (!mbar_wait_warp(&bar->p_full, j & 1, abort)) break;
        if (!mbar_wait_warp(&bar->v_full[s], (j / ST) & 1, abort)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dv = sdesc_sw128(smem_u32(sV + s * C::KVBytes), C::KBox, 1024);
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            if (ks < kNarrow / 16 || !(narrow && j == 0))
              umma_ts(tmem + C::kO, tmem_p + ks * 8, sdesc_at(dv, ks * 2048), idesc_o, (j > 0 || ks > 0));
          umma_commit(&bar->pv_done);
          umma_commit(&bar->v_empty[s]);
        }
      }
    }
  } else if (warp == 5) {
    // ---------------- producer: the K and V tiles past the first ST
    for (int j = ST; j < kl.n; ++j) {
      const int s = j % ST;
      if (!mbar_wait_warp(&bar->k_empty[s], (j / ST - 1) & 1, abort)) break;
      if (elect_one()) load_k(j);
      if (!mbar_wait_warp(&bar->v_empty[s], (j / ST - 1) & 1, abort)) break;
      if (elect_one()) load_v(j);
    }
  } else {
    // ---------------- softmax: warps 0-3, one query row per thread
    const int prow = row0 + warp * 32 + lane;
    const int t_r = prow / kk;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16, lane_base = tmem + lane_off, lane_p = tmem_p + lane_off;
    RowTile st{-INFINITY, 0.f, true};
    for (int j = 0; j < kl.n && st.ok; ++j) {
      const int base = kl.tile(j) * KT;
      // some row does not see some key: one after its token, or one its window has left behind
      const bool border = base + KT - 1 > t_first || (base < t_last - p.window + 1 && base + KT > p.sinks);
      st.ok = mbar_wait_short(&bar->s_full, j & 1, abort);
      tc_fence_after();
      if (narrow && j == 0)
        softmax_tile<D, kNarrow>(st, bar, lane_base, lane_p, j, base, t_r, true, p, abort);
      else
        softmax_tile<D, KT>(st, bar, lane_base, lane_p, j, base, t_r, border, p, abort);
    }
    // ---------------- epilogue: O / l -> bf16
    st.ok = mbar_wait_short(&bar->pv_done, (kl.n - 1) & 1, abort) && st.ok;
    tc_fence_after();
    const bool valid = prow < rows_total && st.ok;
    const float inv_l = 1.f / st.l;
    gqe_bf16_t* orow = (routed ? p.o_routed : p.o_sh) + ((size_t)seq * rows_total + prow) * D;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      tmem_ld32(lane_base + C::kO + c0, o);
      if (valid) {
        uint4* d4 = reinterpret_cast<uint4*>(orow + c0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pk[e] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * e]) * inv_l,
                                __uint_as_float(o[8 * c + 2 * e + 1]) * inv_l);
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
  if (warp == 4) {
    drain_after_abort(abort);      // what is in flight lands before another CTA gets the columns
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
    if (C::kApart) tmem_dealloc(tmem_p, 32);
  }
  report_abort(abort, p.err, kErrTimeoutAttn);
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
