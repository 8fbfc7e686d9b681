// attn_bwd_window.cu -- backward of the windowed prefill attention on tcgen05.
//
// The mathematics is attn_bwd.cu's (dV = P^T dO, dS = scale * P o (dP - Delta),
// dK = dS^T q, dq = dS K with P from the forward's log-sum-exp) over the keys a
// window leaves: query t sees key p when p <= t and (p > t - window or
// p < sinks).  Key tile j therefore walks the query tiles from token 128 j up to
// the last token whose window reaches its last key, and to the end when it
// holds a sink.
//
// Under a window the walks are short (window / 128 + 1 query tiles of each kind
// of row) except the sink tiles', which are as long as the sequence.  One CTA
// per key tile, as without a window, then spends a third of its time starting
// and ending (5.5 of 16.6 us at a window of 512, d = 64) and waits for the sink
// tiles.  Here the walks of all key tiles of all sequences form one list of
// (key tile, query tile) pairs, cut into equal stretches, one or a few per SM,
// and each CTA runs its stretches as one pipeline: the loads and products of the
// next key tile start while the last one's are still running.  A walk cut by a
// stretch's end leaves its dK, dV sums in fp32 in a slot of the stretch, and
// attn_bwd_window_post_kernel adds the slots of a walk in their order, so dK
// and dV do not depend on timing.  dQ goes through TMA reduce-add into fp32 as
// in attn_bwd.cu; with several stretches per CTA all CTAs work on one part of
// the sequences at a time, so that the part's dQ sums stay in L2 (attn_bwd_window_plan:
// up to 256 MB of them in all).
//
// CTA: 512 threads, roles, tensor memory and barriers as in attn_bwd.cu, with
// every ring counted over the whole stretch, but for d = 128: dK reads dS from
// shared memory there, so S^T(i+1) waits only for dV(i), and the drain warps
// take a whole dQ row into registers, so dP^T(i+1) (over dQ(i)'s columns) waits
// less.  d = 64 keeps two key tiles' K and
// V in shared memory; d = 128 has room for one.  Tensor memory holds one dK and
// one dV: the next key tile's first products into them wait until the drain
// warps have read them (acc_free).
//
// Delta = dO . O takes the forward's O, which is rounded to bf16.  The error is
// |dO||O| 2^-9 a row, next to |dO||V - O| in dP - Delta: of no account when O
// averages many keys (|O| is then about |V| / sqrt(n)), but as large as all other
// roundings together for a row that sees two or three (dq of 3-token sequences
// 0.0039 off, norm-wise, against 0.0018 in fp32).  Rows that see at most kFewKeys
// keys take Delta = sum_j P_j dP_j in fp32 instead, in the prep kernel; at nine
// keys what is left is a third of the other roundings, a tenth of their variance.
//
// P and dS are computed with packed pairs (f32x2): the prep kernel stores -LSE2
// and -Delta, so a pair costs one FMA before its exponentials and one add and
// one multiply after them; the scale of dS moves to where dK and dq are rounded.
// What bounds the main kernel is each tile's chain S -> P, dP -> dS -> dQ, dK: 8 x
// 2048 tokens of 9 heads, d = 64, under a 512-token window 102 us (0.24 of the
// measured bf16 rate); 2 x 8192 tokens of 17 heads, d = 128, under 1024 tokens 491
// us (0.42), where tensor memory is full and dP(i+1) waits for dQ(i)'s columns.
// Exponentials on the FMA-pipe polynomial (2 or 4 of 16 pairs) changed the time
// by +0.5 and +2.5 %, so all run on MUFU.
#include "attn.cuh"
#include "launch.cuh"

namespace gqe {

namespace {

constexpr int kThreadsW = 512;
constexpr int kFewKeys = 8;
constexpr int kTileW = 128;
constexpr int kBoxW = 128 * 64 * 2;   // one 128-row x 64-column bf16 TMA box

struct __align__(8) BwdWinBarriers {
  uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2];
  uint64_t q_full[2], q_empty[2], o_full[2], o_empty[2];
  uint64_t s_full, s_free, p_full, pv_done, dp_full, ds_full, dk_done, dq_full, dq_free, acc_free;
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct BwdWinCfg {
  static constexpr int NB = D / 64;
  static constexpr int TileBytes = NB * kBoxW;        // one 128-row tile of Q, dO, K or V
  static constexpr bool kWide = D == 128;
  static constexpr int KVB = kWide ? 1 : 2;           // key tiles whose K and V are held
  static constexpr int OST = kWide ? 1 : 2;           // dO ring depth
  static constexpr int EpiCh = kWide ? 1 : D / 32;    // 32-column dQ chunks staged per warp at once
  static constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 256 + D;
  static constexpr uint32_t kDQ = kWide ? 128 : 384;
  static constexpr uint32_t kPT = 448;                // d = 64: P^T
  static constexpr int OffK = 0;
  static constexpr int OffV = OffK + KVB * TileBytes;
  static constexpr int OffQ = OffV + KVB * TileBytes;           // [2] stages
  static constexpr int OffDO = OffQ + 2 * TileBytes;            // [OST]
  static constexpr int OffDS = OffDO + OST * TileBytes;         // 128 x 128 bf16, MN-major
  static constexpr int OffEpi = OffDS + 2 * kBoxW;              // 4 warps x EpiCh x 4 KB
  static constexpr int OffLse = OffEpi + 4 * EpiCh * 4096;      // [2][128] f32
  static constexpr int OffDelta = OffLse + 2 * 512;             // [2][128] f32
  static constexpr int OffBar = OffDelta + 2 * 512;
  static constexpr size_t Smem = 1024 + OffBar + sizeof(BwdWinBarriers);
  // tensor-memory columns of P^T and (d = 64) dS^T, by 16-query k-step and by warpgroup
  static __device__ __forceinline__ uint32_t pt_col(int ks) { return kWide ? kS + ks * 8 : kPT + ks * 8; }
  static __device__ __forceinline__ uint32_t dst_col(int ks) { return kDP + (ks >> 2) * 64 + (ks & 3) * 8; }
  static __device__ __forceinline__ uint32_t pt_wcol(int w) { return kWide ? kS + 32 * w : kPT + 32 * w; }
  static __device__ __forceinline__ uint32_t dst_wcol(int w) { return kDP + 64 * w; }
};

// Query tiles (routed, then shared) that key tile jt of a group sees.
__host__ __device__ inline void walk_counts(int T, int k, int window, int sinks, int jt, bool shared, int* n_r,
                                            int* n_s) {
  int t_hi = T - 1;                                 // last token that sees a key of the tile
  if (jt * kTileW >= sinks) {
    const int reach = jt * kTileW + kTileW - 2 + window;
    if (reach < t_hi) t_hi = reach;
  }
  *n_r = (int)((unsigned)((t_hi + 1) * k + kTileW - 1) / kTileW) - jt * k;
  *n_s = shared ? (int)((unsigned)t_hi / kTileW) + 1 - jt : 0;
}

// Position in a CTA's stretch: query tile n of the piece [off, off + cnt) of key
// tile jt's walk.
struct Stretch {
  int left;          // query tiles of the stretch from this piece on
  int s, b, g;       // KV sequence, its batch entry and its group
  int jt, off;       // key tile, first query tile of the piece
  int n_r, total;    // routed query tiles and all query tiles of the whole walk
  int cnt, n;        // query tiles of the piece, position in it
  int item;          // pieces before this one
  int id;            // the stretch

  __device__ __forceinline__ void open(const AttnBwdParams& p) {
    int n_s;
    walk_counts(p.T, p.k, p.window, p.sinks, jt, p.n_shared && g == p.sg, &n_r, &n_s);
    total = n_r + n_s;
    cnt = min(total - off, left);
    n = 0;
  }
  __device__ __forceinline__ void load(const AttnBwdParams& p, const AttnBwdSchedule& S) {
    left = S.count[id];
    s = S.seq[id];
    b = s / p.G;
    g = s - b * p.G;
    jt = S.jt[id];
    off = S.off[id];
    open(p);
  }
  __device__ __forceinline__ void start(const AttnBwdParams& p, const AttnBwdSchedule& S) {
    id = blockIdx.x;
    item = 0;
    load(p, S);
  }
  __device__ __forceinline__ bool next(const AttnBwdParams& p, const AttnBwdSchedule& S) {
    if (++n < cnt) return true;
    left -= cnt;
    ++item;
    if (left <= 0) {
      id += S.n_ctas;
      if (id >= S.n_ctas * S.n_rounds) return false;
      load(p, S);
      return true;
    }
    off = 0;
    if (++jt * kTileW >= p.T) {
      jt = 0;
      ++s;
      if (++g == p.G) g = 0, ++b;
    }
    open(p);
    return true;
  }
  __device__ __forceinline__ bool first() const { return n == 0; }
  __device__ __forceinline__ bool last() const { return n == cnt - 1; }
  __device__ __forceinline__ bool whole() const { return off == 0 && cnt == total; }
  // the query tile: of the shared head or not, its index, its first row in the padded row space
  __device__ __forceinline__ bool shared() const { return off + n >= n_r; }
  __device__ __forceinline__ int qi(const AttnBwdParams& p) const {
    return shared() ? jt + off + n - n_r : jt * p.k + off + n;
  }
  __device__ __forceinline__ int row_pad(const AttnBwdParams& p) const {
    return shared() ? p.B * p.G * p.rows_pad + b * p.rows_pad_sh + qi(p) * kTileW
                    : s * p.rows_pad + qi(p) * kTileW;
  }
};

// One product's k-steps, unrolled: rolled they save 10 KB of code but issue
// slower, and the chain S -> P -> dV -> S waits for the issue (train step of 2 x
// 8192 tokens, d = 128: 4.55 against 3.9 us a tile).
// Both operands K-major, D wide (S, dP).
template <int D>
__device__ __forceinline__ void product_kk(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc) {
  const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, 16, 1024);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t off = (ks >> 2) * kBoxW + (ks & 3) * 32;
    umma_ss(acc, sdesc_at(da, off), sdesc_at(db, off), idesc, ks > 0);
  }
}
// A from tensor memory (query k-steps 0-3 at a0, 4-7 at a1, 8 columns each), B
// MN-major in shared memory (dV, dK).
__device__ __forceinline__ void product_ts(uint32_t acc, uint32_t a0, uint32_t a1, uint32_t b, uint32_t idesc,
                                           bool accumulate) {
  const uint64_t db = sdesc_sw128(b, kBoxW, 1024);
#pragma unroll
  for (int ks = 0; ks < kTileW / 16; ++ks)
    umma_ts(acc, (ks < 4 ? a0 : a1) + (ks & 3) * 8, sdesc_at(db, ks * 2048), idesc, accumulate || ks > 0);
}
// A K-major and B MN-major in shared memory (dK at d = 128).
__device__ __forceinline__ void product_km(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, kBoxW, 1024);
#pragma unroll
  for (int ks = 0; ks < kTileW / 16; ++ks)
    umma_ss(acc, sdesc_at(da, (ks >> 2) * kBoxW + (ks & 3) * 32), sdesc_at(db, ks * 2048), idesc,
            accumulate || ks > 0);
}
// Both operands MN-major in shared memory (dQ).
__device__ __forceinline__ void product_mm(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc) {
  const uint64_t da = sdesc_sw128(a, kBoxW, 1024), db = sdesc_sw128(b, kBoxW, 1024);
#pragma unroll
  for (int ks = 0; ks < kTileW / 16; ++ks)
    umma_ss(acc, sdesc_at(da, ks * 2048), sdesc_at(db, ks * 2048), idesc, ks > 0);
}

// One row of a key tile's dK and dV out of tensor memory, then acc_free.  A cut
// walk's go to its slot in fp32 (slot 0 of the stretch when the piece starts
// inside the walk, else slot 1), a whole walk's are rounded.
template <int D>
__device__ __forceinline__ void read_acc(const Stretch& c, const AttnBwdParams& p, uint32_t tmem_lane, int kv,
                                         uint64_t* acc_free) {
  using C = BwdWinCfg<D>;
  const int kv_pos = c.jt * kTileW + kv;
  const bool whole = c.whole();
  float* slot = p.part + ((size_t)(2 * c.id + (c.off > 0 ? 0 : 1)) * 2 * kTileW + kv) * D;
  const size_t orow = ((size_t)c.s * p.T + kv_pos) * D;
#pragma unroll 1
  for (int c0 = 0; c0 < 2 * D; c0 += 32) {       // dK's columns, then dV's
    const bool dv = c0 >= D;
    const int col = dv ? c0 - D : c0;
    uint32_t v[32];
    tmem_ld32(tmem_lane + (dv ? C::kDV : C::kDK) + col, v);
    if (c0 == 2 * D - 32) {
      tc_fence_before();
      mbar_arrive(acc_free);
    }
    if (!whole) {
      uint4* d4 = reinterpret_cast<uint4*>(slot + (dv ? (size_t)kTileW * D : 0) + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) d4[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if (kv_pos < p.T) {
      const float f = dv ? 1.f : p.scale;
      uint4* d4 = reinterpret_cast<uint4*>((dv ? p.dV : p.dK) + orow + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * e]) * f, __uint_as_float(v[8 * i + 2 * e + 1]) * f);
        d4[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsW, 1)
attn_bwd_window_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapQs,
                       const __grid_constant__ CUtensorMap mapdO, const __grid_constant__ CUtensorMap mapdOs,
                       const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                       const __grid_constant__ CUtensorMap mapdQ, const __grid_constant__ AttnBwdParams p,
                       const __grid_constant__ AttnBwdSchedule sched) {
  using C = BwdWinCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sDS = smem + C::OffDS;
  float* sLse = reinterpret_cast<float*>(smem + C::OffLse);
  float* sDelta = reinterpret_cast<float*>(smem + C::OffDelta);
  BwdWinBarriers* bar = reinterpret_cast<BwdWinBarriers*>(smem + C::OffBar);
  volatile int* abort = &bar->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](uint64_t* b, uint32_t parity) { return mbar_wait_short(b, parity & 1, abort); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->k_empty[i], 2);        // the last S and the last dQ of the key tile
      mbar_init(&bar->v_empty[i], 1);        // the last dP
      mbar_init(&bar->q_full[i], 1);
      mbar_init(&bar->q_empty[i], 2 + 256);
      mbar_init(&bar->o_full[i], 1);
      mbar_init(&bar->o_empty[i], 1);
    }
    mbar_init(&bar->s_full, 1);
    mbar_init(&bar->s_free, 256);
    mbar_init(&bar->p_full, 256);
    mbar_init(&bar->pv_done, 1);
    mbar_init(&bar->dp_full, 1);
    mbar_init(&bar->ds_full, 256);
    mbar_init(&bar->dk_done, 1);
    mbar_init(&bar->dq_full, 1);
    mbar_init(&bar->dq_free, 128);
    mbar_init(&bar->acc_free, 128);
    bar->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapQ);
    tma_prefetch_desc(&mapdO);
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
    tma_prefetch_desc(&mapdQ);
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  pdl_launch_dependents();
  pdl_wait();

  Stretch c;
  c.start(p, sched);

  // registers per thread, adding up to the launch's 512 x 128: issue, softmax and
  // drain warps 96 x 128 + 144 x 256 + 128 x 128; at d = 128, where a drain warp
  // holds a whole dQ row, 80 x 128 + 136 x 256 + 160 x 128
  if (warp < 4) {
    set_regs_down<C::kWide ? 80 : 96>();
    auto wait_w = [&](uint64_t* b, uint32_t parity) { return mbar_wait_warp(b, parity & 1, abort); };
    const bool leader = elect_one();
    if (warp == 0) {
      // ---------------- producer: K, V of each key tile; Q, dO, -LSE2, -Delta of each query tile
      uint32_t N = 0;
      do {
        if (c.first()) {
          const int b = c.item % C::KVB;
          const uint32_t ph = c.item / C::KVB - 1;
          if (c.item >= C::KVB && !wait_w(&bar->k_empty[b], ph)) break;
          if (leader) {
            mbar_arrive_expect_tx(&bar->k_full[b], C::TileBytes);
            for (int bx = 0; bx < C::NB; ++bx)
              tma_load_3d(smem + C::OffK + b * C::TileBytes + bx * kBoxW, &mapK, &bar->k_full[b], bx * 64,
                          c.jt * kTileW, c.s);
          }
          if (c.item >= C::KVB && !wait_w(&bar->v_empty[b], ph)) break;
          if (leader) {
            mbar_arrive_expect_tx(&bar->v_full[b], C::TileBytes);
            for (int bx = 0; bx < C::NB; ++bx)
              tma_load_3d(smem + C::OffV + b * C::TileBytes + bx * kBoxW, &mapV, &bar->v_full[b], bx * 64,
                          c.jt * kTileW, c.s);
          }
        }
        const int st = N & 1, so = N % C::OST;
        const bool shr = c.shared();
        const CUtensorMap* mq = shr ? &mapQs : &mapQ;
        const CUtensorMap* mo = shr ? &mapdOs : &mapdO;
        const int seq = shr ? c.b : c.s, row = c.qi(p) * kTileW, rp = c.row_pad(p);
        if (N >= 2 && !wait_w(&bar->q_empty[st], (N >> 1) - 1)) break;
        if (leader) {
          mbar_arrive_expect_tx(&bar->q_full[st], C::TileBytes + 2 * 512);
          for (int bx = 0; bx < C::NB; ++bx)
            tma_load_3d(smem + C::OffQ + st * C::TileBytes + bx * kBoxW, mq, &bar->q_full[st], bx * 64, row, seq);
          bulk_load(sLse + st * 128, p.lse2 + rp, 512, &bar->q_full[st]);
          bulk_load(sDelta + st * 128, p.delta + rp, 512, &bar->q_full[st]);
        }
        if (N >= C::OST && !wait_w(&bar->o_empty[so], N / C::OST - 1)) break;
        if (leader) {
          mbar_arrive_expect_tx(&bar->o_full[so], C::TileBytes);
          for (int bx = 0; bx < C::NB; ++bx)
            tma_load_3d(smem + C::OffDO + so * C::TileBytes + bx * kBoxW, mo, &bar->o_full[so], bx * 64, row, seq);
        }
        ++N;
      } while (c.next(p, sched));
    } else if (warp == 1) {
      // ---------------- MMA issuer A: S^T, dP^T, dV
      constexpr uint32_t idesc_s = idesc_bf16_f32(kTileW, kTileW, false, false);
      constexpr uint32_t idesc_v = idesc_bf16_f32(kTileW, D, false, true);
      auto issue_s = [&](const Stretch& t, uint32_t N) {
        const int st = N & 1, b = t.item % C::KVB;
        if (t.first() && !wait_w(&bar->k_full[b], t.item / C::KVB)) return false;
        if (!wait_w(&bar->q_full[st], N >> 1)) return false;
        tc_fence_after();
        if (leader) {
          product_kk<D>(tmem + C::kS, smem_u32(smem + C::OffK + b * C::TileBytes),
                        smem_u32(smem + C::OffQ + st * C::TileBytes), idesc_s);
          umma_commit(&bar->s_full);
          if (t.last()) umma_commit(&bar->k_empty[b]);
        }
        return true;
      };
      // nx is query tile N + 1, c query tile N (the first round has none)
      Stretch nx = c;
      bool more = true;
      for (uint32_t N = 0xFFFFFFFFu;; ++N) {
        const bool none = N == 0xFFFFFFFFu;
        // d = 64: S^T(N+1) as soon as the warpgroups hold S^T(N) in registers
        if (!C::kWide && more) {
          if (!none && !wait_w(&bar->s_free, N)) break;
          if (!issue_s(nx, N + 1)) break;
        }
        if (!none) {
          // dV += P^T dO_i once P^T is in tensor memory (and, at a key tile's
          // first query tile, the last key tile's dV has been read)
          if (!wait_w(&bar->p_full, N)) break;
          if (c.first() && c.item > 0 && !wait_w(&bar->acc_free, c.item - 1)) break;
          tc_fence_after();
          if (leader) {
            product_ts(tmem + C::kDV, tmem + C::pt_col(0), tmem + C::pt_col(4),
                       smem_u32(smem + C::OffDO + (N % C::OST) * C::TileBytes), idesc_v, !c.first());
            umma_commit(&bar->pv_done);
            umma_commit(&bar->q_empty[N & 1]);
            umma_commit(&bar->o_empty[N % C::OST]);
          }
          if (!more) break;
          // d = 64: dP^T(N+1) overwrites dS^T(N).  d = 128: S^T(N+1) overwrites
          // P^T(N), dP^T(N+1) overwrites dQ(N)
          if (!wait_w(C::kWide ? &bar->pv_done : &bar->dk_done, N)) break;
        }
        if (C::kWide) {
          if (!issue_s(nx, N + 1)) break;
          if (!none && !wait_w(&bar->dq_free, N)) break;
        }
        const int so = (N + 1) % C::OST, b = nx.item % C::KVB;
        if (nx.first() && !wait_w(&bar->v_full[b], nx.item / C::KVB)) break;
        if (!wait_w(&bar->o_full[so], (N + 1) / C::OST)) break;
        tc_fence_after();
        if (leader) {
          product_kk<D>(tmem + C::kDP, smem_u32(smem + C::OffV + b * C::TileBytes),
                        smem_u32(smem + C::OffDO + so * C::TileBytes), idesc_s);
          umma_commit(&bar->dp_full);
          if (nx.last()) umma_commit(&bar->v_empty[b]);
        }
        c = nx;
        more = nx.next(p, sched);
      }
    } else if (warp == 2) {
      // ---------------- MMA issuer B: dK += dS^T Q_i, dQ_i = dS K_j
      constexpr uint32_t idesc_k = idesc_bf16_f32(kTileW, D, false, true);
      constexpr uint32_t idesc_q = idesc_bf16_f32(kTileW, D, true, true);
      uint32_t N = 0;
      do {
        const int b = c.item % C::KVB;
        if (!wait_w(&bar->ds_full, N)) break;
        tc_fence_after();
        const uint32_t q0 = smem_u32(smem + C::OffQ + (N & 1) * C::TileBytes);
        const uint32_t k0 = smem_u32(smem + C::OffK + b * C::TileBytes);
        if (C::kWide) {
          // dQ first: its drain is what dP^T(N+1) waits for (dQ sits over dP^T's
          // columns, which the warpgroups have read, ds_full)
          if (leader) {
            product_mm(tmem + C::kDQ, smem_u32(sDS), k0, idesc_q);
            umma_commit(&bar->dq_full);
          }
          if (c.first() && c.item > 0 && !wait_w(&bar->acc_free, c.item - 1)) break;
          tc_fence_after();
          if (leader) {
            product_km(tmem + C::kDK, smem_u32(sDS), q0, idesc_k, !c.first());
            umma_commit(&bar->q_empty[N & 1]);
            umma_commit(&bar->dk_done);
          }
        } else {
          if (c.first() && c.item > 0 && !wait_w(&bar->acc_free, c.item - 1)) break;
          tc_fence_after();
          if (leader) {
            product_ts(tmem + C::kDK, tmem + C::dst_col(0), tmem + C::dst_col(4), q0, idesc_k, !c.first());
            umma_commit(&bar->q_empty[N & 1]);
            umma_commit(&bar->dk_done);      // dS^T(N) has been read from tensor memory
          }
          // dQ(N) over dQ(N-1): wait for its drain
          if (N >= 1 && !wait_w(&bar->dq_free, N - 1)) break;
          tc_fence_after();
          if (leader) {
            product_mm(tmem + C::kDQ, smem_u32(sDS), k0, idesc_q);
            umma_commit(&bar->dq_full);
          }
        }
        if (leader && c.last()) umma_commit(&bar->k_empty[b]);
        ++N;
      } while (c.next(p, sched));
    }
  } else if (warp < 12) {
    set_regs_up<C::kWide ? 136 : 144>();
    // ---------------- P and dS: one key row per thread, 64 query columns per warpgroup
    const int wg = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t col0 = (uint32_t)(wg * 64);
    const unsigned long long sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
    uint32_t N = 0;
    // d = 128: a thread whose wait failed goes on to the next tile's vote, where all of
    // the two warpgroups leave together; the others would wait for it there
    bool ok = true;
    do {
      const int st = N & 1;
      const int kv_pos = c.jt * kTileW + r, kk = c.shared() ? 1 : p.k, base = c.qi(p) * kTileW + (int)col0;
      // query columns c < cmin belong to tokens before this key, c >= cmax to
      // tokens whose window starts behind it
      const int cmin = kv_pos * kk - base;
      const int cmax = kv_pos < p.sinks ? kTileW : (kv_pos + p.window) * kk - base;
      ok = ok && wait(&bar->q_full[st], N >> 1) && wait(&bar->s_full, N);
      if (!C::kWide && !ok) break;
      tc_fence_after();
      const float* lse2 = sLse + st * 128 + col0;
      const float* dlt = sDelta + st * 128 + col0;
      float pf[64];
      if (ok) {
        tmem_ld64(tmem + lane_off + C::kS + col0, reinterpret_cast<uint32_t*>(pf));
        if (!C::kWide) {
          tc_fence_before();
          mbar_arrive(&bar->s_free);      // S^T(N) is in registers
        }
#pragma unroll
        for (int q = 0; q < 64; q += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(lse2 + q);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(pf[q + e], pf[q + e + 1]), sl2x2, e ? f2_pack(l4.z, l4.w) : f2_pack(l4.x, l4.y)),
                      x0, x1);
            pf[q + e] = ex2(x0);
            pf[q + e + 1] = ex2(x1);
          }
        }
        if (cmin > 0 || cmax < 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t vis = ~bits_below(cmin, 32 * h) & bits_below(cmax, 32 * h);
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (!((vis >> q) & 1u)) pf[32 * h + q] = 0.f;
          }
        }
      }
      if (!C::kWide) {
        // P^T(N-1) must have been read by dV(N-1) before P^T(N) replaces it
        if (N > 0 && !wait(&bar->pv_done, N - 1)) break;
        tc_fence_after();
      } else {
        // both warpgroups hold their S^T columns in registers before warpgroup 1
        // writes P^T over warpgroup 0's
        if (bar_or<1, 256>(!ok)) break;
      }
      {
        uint32_t pk[32];
#pragma unroll
        for (int q = 0; q < 32; ++q) pk[q] = pack_bf16x2(pf[2 * q], pf[2 * q + 1]);
        tmem_st32(tmem + lane_off + C::pt_wcol(wg), pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bar->p_full);

      ok = wait(&bar->dp_full, N);
      if (!ok) {
        if (C::kWide) continue;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t dp[32], dsk[16];
        tmem_ld32(tmem + lane_off + C::kDP + col0 + ch * 32, dp);
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          const int q = ch * 32 + c4 * 4;
          const float4 d4 = *reinterpret_cast<const float4*>(dlt + q);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const unsigned long long t =
                f2_add(f2_pack(__uint_as_float(dp[c4 * 4 + e]), __uint_as_float(dp[c4 * 4 + e + 1])),
                       e ? f2_pack(d4.z, d4.w) : f2_pack(d4.x, d4.y));
            float a0, a1;
            f2_unpack(f2_mul(f2_pack(pf[q + e], pf[q + e + 1]), t), a0, a1);
            dsk[c4 * 2 + e / 2] = pack_bf16x2(a0, a1);
          }
        }
        // d = 64: dS^T row r for dK into this warpgroup's tensor-memory columns
        if (!C::kWide) tmem_st16(tmem + lane_off + C::dst_wcol(wg) + ch * 16, dsk);
        // for dQ (MN-major) and, at d = 128, dK (K-major) into shared memory: the
        // 64-query atom of this warpgroup, 16-byte pieces swizzled by key row, once
        // the last products have read the previous tile's (the second of dQ and dK)
        if (ch == 0 && N > 0) ok = wait(C::kWide ? &bar->dk_done : &bar->dq_full, N - 1);
        if (!ok) break;
        uint8_t* atom = sDS + wg * kBoxW + r * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_shared_v4(atom + (((ch * 4 + j) ^ (r & 7)) << 4), dsk[j * 4], dsk[j * 4 + 1], dsk[j * 4 + 2],
                       dsk[j * 4 + 3]);
      }
      if (!ok) {
        if (C::kWide) continue;
        break;
      }
      if (!C::kWide) tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bar->ds_full);
      mbar_arrive(&bar->q_empty[st]);
      ++N;
    } while (c.next(p, sched));
  } else {
    if (C::kWide) set_regs_up<160>();
    // ---------------- dQ drain (TMA reduce-add into fp32); dK, dV at the end of each key tile
    const int qd = warp & 3;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    uint8_t* stage = smem + C::OffEpi + qd * C::EpiCh * 4096;
    uint32_t N = 0;
    do {
      // dq_full comes first, at a key tile's last query tile too.  These warps wait for
      // dk_done and pv_done only there, and a wait's parity means phase N only once
      // phase N-1 is over, which dq_full(N) implies: the warps that made dS(N) had
      // passed pv_done(N-1) (d = 64) or dk_done(N-1) (d = 128), and dP(N) or S(N) was
      // issued behind the other one.  (Phase N+1 waits for acc_free.)
      if (!wait(&bar->dq_full, N)) break;
      tc_fence_after();
      // A key tile's last query tile: dK and dV first at d = 64, so that the next key
      // tile's products into them start; at d = 128 the next dP^T waits for the dQ
      // drain, so that comes first.
#pragma unroll 1
      for (int step = 0; step < 2; ++step) {
        if ((step == 0) != C::kWide) {
          if (!c.last()) continue;
          if (!wait(&bar->dk_done, N) || !wait(&bar->pv_done, N)) goto out;
          tc_fence_after();
          read_acc<D>(c, p, tmem + lane_off, qd * 32 + lane, &bar->acc_free);
          continue;
        }
        const int row_pad = c.row_pad(p);
        // the whole row at once, so that the columns are free again soon (d = 128:
        // dP^T(N+1) waits for them)
        uint32_t v[D];
        tmem_ld<D>(tmem + lane_off + C::kDQ, v);
        tc_fence_before();
        mbar_arrive(&bar->dq_free);
#pragma unroll
        for (int g0 = 0; g0 < D / 32; g0 += C::EpiCh) {
          // staging free: every earlier reduce of this warp has read it
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::EpiCh; ++i) {
            const uint32_t* w = v + (g0 + i) * 32;
            uint8_t* rowp = stage + i * 4096 + lane * 128;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(rowp + ((j ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < C::EpiCh; ++i)
              tma_reduce_add_2d(&mapdQ, stage + i * 4096, (g0 + i) * 32, row_pad + qd * 32);
            bulk_commit();
          }
        }
      }
      ++N;
    } while (c.next(p, sched));
  out:
    if (lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    drain_after_abort(abort);      // what is in flight lands before another CTA gets the columns
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  report_abort(abort, p.err, kErrTimeoutAttnBwd);
}

__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
  float d = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) d += bf16_lo(av[e]) * bf16_lo(bv[e]) + bf16_hi(av[e]) * bf16_hi(bv[e]);
  return d;
}

// The tokens of a sequence that see at most kFewKeys keys: the first ones, since
// token t sees min(t + 1, ...) of them and never fewer than token t - 1.
__host__ __device__ __forceinline__ int few_key_tokens(int T, int window, int sinks) {
  return T <= kFewKeys || (long long)window + sinks <= kFewKeys ? T : kFewKeys;
}

// Delta of a row that sees at most kFewKeys keys, sum_j P_j dP_j, by one warp:
// d/8 lanes a key, the loads of 64 / (d/8) keys in flight.  No shared memory: a
// kernel that has 32 bytes of it makes the SMs set their L1 split anew between
// the attention kernels around it, 8 us of a 42 us step.
__device__ __forceinline__ void few_keys_delta(const AttnBwdParams& p, int n_few, int tokens) {
  const int tpr = p.d / 8, lane = threadIdx.x & 31, part = lane % tpr, at_once = 32 / tpr;
  int q = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (q >= n_few) return;
  const int BG = p.B * p.G;
  const bool shared = q >= BG * tokens * p.k;
  if (shared) q -= BG * tokens * p.k;
  const int kk = shared ? 1 : p.k;
  const int sq = q / (tokens * kk), r = q - sq * tokens * kk;
  const int t = r / kk, lo = max(0, t - p.window + 1), first = min(p.sinks, lo), n = first + t - lo + 1;
  const long long src = (long long)sq * p.T * kk + r;
  const long long kv0 = (long long)(shared ? sq * p.G + p.sg : sq) * p.T * tpr + part;
  const uint4 qv = reinterpret_cast<const uint4*>((shared ? p.q_sh : p.q_routed) + src * p.d)[part];
  const uint4 dov = reinterpret_cast<const uint4*>((shared ? p.do_sh : p.do_routed) + src * p.d)[part];
  const float lse2 = p.lse[shared ? (long long)BG * p.T * p.k + src : src] * 1.4426950408889634f;
  float delta = 0.f;
  for (int j0 = lane / tpr; j0 < kFewKeys; j0 += 2 * at_once) {
    float s[2], dp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = min(j0 + i * at_once, n - 1);
      const long long at = kv0 + (long long)(j < first ? j : lo + j - first) * tpr;
      s[i] = dot8(qv, reinterpret_cast<const uint4*>(p.K)[at]);
      dp[i] = dot8(dov, reinterpret_cast<const uint4*>(p.V)[at]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      for (int off = tpr >> 1; off > 0; off >>= 1) {
        s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], off);
        dp[i] += __shfl_xor_sync(0xFFFFFFFFu, dp[i], off);
      }
      if (j0 + i * at_once < n) delta = fmaf(ex2(fmaf(s[i], p.scale_log2, -lse2)), dp[i], delta);
    }
  }
  for (int off = tpr; off < 32; off <<= 1) delta += __shfl_xor_sync(0xFFFFFFFFu, delta, off);
  if (lane == 0)
    p.delta[(shared ? (long long)BG * p.rows_pad : 0) + (long long)sq * (shared ? p.rows_pad_sh : p.rows_pad) + r] =
        -delta;
}

// -Delta and -LSE2 of every row of the padded row space (LSE2 +inf and Delta 0
// on padding rows, so their P is 0), and the dQ accumulator zeroed.  d/8 threads
// a row, 16 bytes each; HBM-bound (o, dO, the accumulator).  The first
// few_blocks blocks are few_keys_delta's instead: in the rows' own threads, one
// key after the other, it was 12 us of a 160 us step, by its latency and by the
// registers that took the other rows' occupancy (six blocks an SM, 40 registers
// and a few spills in few_keys_delta, against 51 registers: 2 % of that step).
// When all rows are few_keys_delta's (window + sinks <= kFewKeys) they are 75 us
// of a 174 us step of the same size, the price of their Delta.
__global__ void __launch_bounds__(256, 6) attn_bwd_window_prep_kernel(const __grid_constant__ AttnBwdParams p,
                                                                   int few_blocks, int few_tokens) {
  pdl_launch_dependents();
  pdl_wait();
  if ((int)blockIdx.x < few_blocks) {
    few_keys_delta(p, p.B * few_tokens * (p.G * p.k + p.n_shared), few_tokens);
    return;
  }
  const int log_tpr = p.d == 64 ? 3 : 4, tpr = 1 << log_tpr, part = threadIdx.x & (tpr - 1);
  const int pr = (int)(blockIdx.x - few_blocks) * (256 >> log_tpr) + (threadIdx.x >> log_tpr);   // fewer than 2^31 rows
  if (pr >= (int)p.n_rows_pad) return;      // whole rows: tpr divides 32
  const unsigned row_lanes = (tpr == 8 ? 0xFFu : 0xFFFFu) << (threadIdx.x & 31 & ~(tpr - 1));
  const int BG = p.B * p.G;
  const int routed_rows = BG * p.rows_pad;
  const bool shared = pr >= routed_rows;
  const int q2 = shared ? pr - routed_rows : pr;
  const int pad = shared ? p.rows_pad_sh : p.rows_pad, kk = shared ? 1 : p.k;
  const int sq = q2 / pad, r = q2 - sq * pad;       // sequence (or batch entry), row in it
  const bool valid = r < p.T * kk;
  const long long src = (long long)sq * p.T * kk + r;
  const gqe_bf16_t* o = (shared ? p.o_sh : p.o_routed) + src * p.d;
  const gqe_bf16_t* dO = (shared ? p.do_sh : p.do_routed) + src * p.d;
  float lse2 = INFINITY, delta = 0.f;
  if (valid) {
    lse2 = p.lse[shared ? (long long)BG * p.T * p.k + src : src] * 1.4426950408889634f;
    delta = dot8(reinterpret_cast<const uint4*>(o)[part], reinterpret_cast<const uint4*>(dO)[part]);
    for (int off = tpr >> 1; off > 0; off >>= 1) delta += __shfl_xor_sync(row_lanes, delta, off);
  }
  float4* acc = reinterpret_cast<float4*>(p.dq_acc + (size_t)pr * p.d + part * 8);
  acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
  acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (part == 0) {
    if (!valid || r >= few_tokens * kk) p.delta[pr] = -delta;
    p.lse2[pr] = -lse2;
  }
}

// dK, dV of a walk that the stretches' ends cut: the pieces of the walk cut
// between stretches c-1 and c added in their order, when that is the walk's
// first cut.
// Each of the kJoinBlocks blocks takes its part of the tile.
constexpr int kJoinBlocks = 16;
__device__ __forceinline__ void join_walk(const AttnBwdParams& p, const AttnBwdSchedule& S, int c, int block) {
  const int s = S.seq[c], jt = S.jt[c];
  if (S.off[c] == 0) return;                                                     // the walk starts here
  if (S.seq[c - 1] == s && S.jt[c - 1] == jt && S.off[c - 1] > 0) return;         // cut before
  int last = c;
  const int n = S.n_ctas * S.n_rounds;
  while (last + 1 < n && S.seq[last + 1] == s && S.jt[last + 1] == jt && S.off[last + 1] > 0) ++last;
  const size_t slot = (size_t)2 * kTileW * p.d;
  const int per = p.d / 4;
  for (int e = block * 256 + threadIdx.x; e < 2 * kTileW * per; e += kJoinBlocks * 256) {
    const int c4 = e % per, row = e / per % kTileW, which = e / per / kTileW;
    const int kv_pos = jt * kTileW + row;
    if (kv_pos >= p.T) continue;
    const size_t at = ((size_t)which * kTileW + row) * p.d + c4 * 4;
    float4 a = *reinterpret_cast<const float4*>(p.part + (size_t)(2 * (c - 1) + 1) * slot + at);
#pragma unroll 4
    for (int i = c; i <= last; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(p.part + (size_t)(2 * i) * slot + at);
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
    const float f = which ? 1.f : p.scale;
    gqe_bf16_t* dst = (which ? p.dV : p.dK) + ((size_t)s * p.T + kv_pos) * p.d;
    reinterpret_cast<uint2*>(dst)[c4] = make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
  }
}

// The first (stretches - 1) * kJoinBlocks blocks join the cut walks, the others
// round dq from its fp32 sums (d/8 threads a row, valid rows only).
__global__ void __launch_bounds__(256)
attn_bwd_window_post_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ AttnBwdSchedule S) {
  pdl_launch_dependents();
  pdl_wait();
  const int n_join = (S.n_ctas * S.n_rounds - 1) * kJoinBlocks;
  if ((int)blockIdx.x < n_join) {
    join_walk(p, S, blockIdx.x / kJoinBlocks + 1, blockIdx.x % kJoinBlocks);
    return;
  }
  const int log_tpr = p.d == 64 ? 3 : 4, part = threadIdx.x & ((1 << log_tpr) - 1);
  const int pr = (int)(blockIdx.x - n_join) * (256 >> log_tpr) + (threadIdx.x >> log_tpr);
  const int routed_rows = p.B * p.G * p.rows_pad;
  if (pr >= (int)p.n_rows_pad) return;
  gqe_bf16_t* dst;
  if (pr < routed_rows) {
    const int sq = pr / p.rows_pad, r = pr - sq * p.rows_pad;
    if (r >= p.T * p.k) return;
    dst = p.dq_routed + ((long long)sq * p.T * p.k + r) * p.d;
  } else {
    const int b = (pr - routed_rows) / p.rows_pad_sh, r = pr - routed_rows - b * p.rows_pad_sh;
    if (r >= p.T) return;
    dst = p.dq_sh + ((long long)b * p.T + r) * p.d;
  }
  const float4* a = reinterpret_cast<const float4*>(p.dq_acc + (size_t)pr * p.d + part * 8);
  const float4 x = a[0], y = a[1];
  const float f = p.scale;
  reinterpret_cast<uint4*>(dst)[part] = make_uint4(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f),
                                                   pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
}

}  // namespace

// Walks in the order of the sequences, and of the key tiles in each, cut into
// stretches of equal length (to within one query tile).  One round of stretches
// unless dQ's fp32 sums would not stay in L2: every query tile is added to about
// window / 128 + 2 times, from DRAM if all sequences are worked on at once (2 x
// 8192 tokens, 17 heads of d = 128, 143 MB of sums: 3.3 GB of DRAM traffic in one
// round), so rounds of at most 64 MB of sums, while a stretch keeps 16 query
// tiles (a cut costs two fp32 tiles written and read): 0.87 GB, 556 -> 491 us.  There
// are at most kBwdWindowRounds = 4 rounds, so with more than 256 MB of sums a round's
// are more than 64 MB; what that costs is not measured.
// Parts of the batch in launches of their own, so that the sums are zeroed and
// rounded in L2 too, lost to this by their ramps (760 against 746 us a step).
constexpr long long kRoundBytes = 64 << 20;

void attn_bwd_window_plan(int B, int T, int G, int k, int n_shared, int sg, int d, int window, int sinks,
                          AttnBwdSchedule* S, size_t* off_part, size_t* bytes) {
  const int n_jt = (T + kTileW - 1) / kTileW;
  long long plain = 0, extra = 0;      // query tiles of a sequence's walks: routed, and the shared head's
  for (int j = 0; j < n_jt; ++j) {
    int r, s;
    walk_counts(T, k, window, sinks, j, n_shared != 0, &r, &s);
    plain += r;
    extra += s;
  }
  const long long per_b = plain * G + extra, total = per_b * B;
  AttnBwdLayout L;
  attn_bwd_layout(B, T, G, k, n_shared, d, &L);
  const int ctas = total < kBwdWindowCtas ? (int)total : kBwdWindowCtas;
  int rounds = (int)((L.n_rows_pad * d * 4 + kRoundBytes - 1) / kRoundBytes);
  if (rounds > kBwdWindowRounds) rounds = kBwdWindowRounds;
  while (rounds > 1 && total / ((long long)ctas * rounds) < 16) --rounds;
  const int n = ctas * rounds;
  S->n_ctas = ctas;
  S->n_rounds = rounds;
  int seq = -1, j = 0;
  long long before = 0;                // query tiles before walk (seq, j)
  for (int c = 0; c < n; ++c) {
    const long long at = total * c / n;
    S->count[c] = (int)(total * (c + 1) / n - at);
    // the sequence by division, the key tile by walking (on from the last CTA's)
    const long long b = at / per_b, in_b = at % per_b;
    long long g, base;
    if (in_b < plain * sg) g = in_b / plain, base = g * plain;
    else if (in_b < plain * (sg + 1) + extra) g = sg, base = plain * sg;
    else g = (in_b - extra) / plain, base = g * plain + extra;
    if (b * G + g != seq) {
      seq = (int)(b * G + g);
      j = 0;
      before = b * per_b + base;
    }
    for (;; ++j) {
      int r, s;
      walk_counts(T, k, window, sinks, j, n_shared && g == sg, &r, &s);
      if (at < before + r + s) break;
      before += r + s;
    }
    S->seq[c] = seq;
    S->jt[c] = j;
    S->off[c] = (int)(at - before);
  }
  *off_part = (L.bytes + 255) & ~size_t(255);
  *bytes = *off_part + (size_t)2 * n * 2 * kTileW * d * sizeof(float);
}

template <int D>
static cudaError_t launch_win(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mdO,
                              const CUtensorMap& mdOs, const CUtensorMap& mK, const CUtensorMap& mV,
                              const CUtensorMap& mdQ, const AttnBwdParams& p, const AttnBwdSchedule& S,
                              cudaStream_t stream) {
  auto kern = attn_bwd_window_kernel<D>;
  const size_t smem = BwdWinCfg<D>::Smem;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(S.n_ctas), dim3(kThreadsW), smem, stream, 1, mQ, mQs, mdO, mdOs, mK, mV, mdQ, p, S);
}

cudaError_t launch_attn_bwd_window(const CUtensorMap& mQ, const CUtensorMap& mQs, const CUtensorMap& mdO,
                                   const CUtensorMap& mdOs, const CUtensorMap& mK, const CUtensorMap& mV,
                                   const CUtensorMap& mdQ, const AttnBwdParams& p, const AttnBwdSchedule& S,
                                   cudaStream_t stream) {
  const long long row_blocks = (p.n_rows_pad * (p.d / 8) + 255) / 256;
  const int few_tokens = few_key_tokens(p.T, p.window, p.sinks);
  const int few_blocks = (p.B * few_tokens * (p.G * p.k + p.n_shared) + 7) / 8;
  cudaError_t e = launch_kernel(attn_bwd_window_prep_kernel, dim3((unsigned)(row_blocks + few_blocks)), dim3(256), 0,
                                stream, 1, p, few_blocks, few_tokens);
  if (e != cudaSuccess) return e;
  e = p.d == 64 ? launch_win<64>(mQ, mQs, mdO, mdOs, mK, mV, mdQ, p, S, stream)
                : launch_win<128>(mQ, mQs, mdO, mdOs, mK, mV, mdQ, p, S, stream);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_bwd_window_post_kernel,
                       dim3((unsigned)(row_blocks + (S.n_ctas * S.n_rounds - 1) * kJoinBlocks)), dim3(256), 0, stream,
                       1, p, S);
}

}  // namespace gqe
