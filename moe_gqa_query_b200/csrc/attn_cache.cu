// attn_cache.cu -- attention of a few query tokens per sequence against a dense
// [B, G, L_max, d] cache: a tree of drafted tokens (gqe_attn_tree) and one new
// token under a sliding window (gqe_attn_decode_window); and the move of
// accepted drafted rows into the cache (gqe_cache_commit).
//
// Drafted token i of a sequence sits at position cache_len + depth(i).  With
// window W and S sinks its rows see cache key p when p < cache_len and
// (p > cache_len + depth(i) - W or p < S), and of the drafted tokens its
// ancestors and itself under the same rule.  o = softmax(q K^T * scale) V over
// all of these at once: the cache's key tiles and the tree's are one list.
//
// The T*k routed rows of a group, and the shared head's T rows when the group
// is the shared head's, are packed into 128-row query tiles, so each key tile
// is read once for all of them.  Work item: one query tile of one (b, g) and a
// share of its key list; the shares' softmax states (max, sum, unnormalised O,
// fp32) are joined by attn_cache_merge_kernel.
//
// Per CTA (192 threads, two CTAs per SM): warp 4 brings K tiles by TMA and
// issues S = Q K^T, warp 5 brings V tiles and issues O += P V (P from tensor
// memory), warps 0-3 do the softmax.  Key tiles are 128 keys at d = 64 and 64
// keys at d = 128, so that S, P and O fit 256 tensor-memory columns.
//
// Few rows: a tensor-memory lane is one row and a warp reaches only its own 32
// lanes, so with at most 32 (or 64) rows the softmax of a tile would fall to
// one warp (two).  The rows are repeated in the lanes instead, 4 (or 2) times,
// and repeat q takes the q-th quarter (half) of every tile's keys: P of the
// other keys stays 0 in its lanes.  The repeats are joined like shares, in
// shared memory, at the end.
//
// Keys no row sees (past the lengths, or between the sinks and the first
// row's window) may hold anything: their scores are masked by selection and
// their V rows are zeroed in shared memory before P V reads them.
#include "attn.cuh"
#include "launch.cuh"

namespace gqe {

namespace {

constexpr int kRowsQ = 128;       // query rows per tile
constexpr int kCacheThreads = 192;
constexpr int kCacheST = 2;       // K/V ring depth
constexpr float kCacheRescaleLog2 = 8.0f;

template <int D>
struct CacheCfg {
  static constexpr int NB = D / 64;
  static constexpr int KT = D == 64 ? 128 : 64;          // keys per tile
  static constexpr int QBox = kRowsQ * 128;              // 128 rows x 64 bf16
  static constexpr int KBox = KT * 128;
  static constexpr int QBytes = NB * QBox;
  static constexpr int KVBytes = NB * KBox;
  static constexpr uint32_t kS = 0, kP = KT, kO = D == 64 ? 192 : 128;
  static constexpr int OPitch = D + 4;                   // floats per staged O row
};

struct __align__(16) CacheShared {
  uint32_t anc[2][kMaxTree][4];      // ancestor bits (double-buffered while they are built)
  int up[2][kMaxTree];               // pointer doubling: 2^r levels up, -1 past the root
  int depth[2][kMaxTree];
  float m[kRowsQ], l[kRowsQ];
  uint64_t k_full[kCacheST], k_empty[kCacheST], v_full[kCacheST], v_empty[kCacheST];
  uint64_t s_full, s_free, p_full, pv_done;
  uint32_t tmem_base;
  int abort;
};

template <int D>
constexpr size_t cache_smem() {
  return 1024 + CacheCfg<D>::QBytes + 2 * kCacheST * CacheCfg<D>::KVBytes + sizeof(CacheShared);
}

// One sequence's keys as this query tile's list of key tiles.
struct CacheList {
  int len;           // cache rows
  int m;             // live drafted tokens (1 for a decode step)
  int base;          // position of a row at depth 0
  int lo0;           // first cache row in the window of depth 0
  int n_sink, w0;    // cache tiles 0 .. n_sink-1, then w0, w0+1, ...
  int n_cache, n;    // cache tiles, all tiles (then the tree's)
  template <int KT>
  __device__ __forceinline__ int row(int i) const {   // first row of tile i, in the cache or in the tree
    return (i < n_sink ? i : i < n_cache ? w0 + i - n_sink : i - n_cache) * KT;
  }
};

template <int KT>
__device__ __forceinline__ CacheList cache_list(const CacheAttnParams& p, int b) {
  CacheList c;
  c.len = min(max(p.cache_len[b], 0), p.L_max);
  c.m = !p.tree ? 1 : min(max(p.tree_len ? p.tree_len[b] : p.T, 0), p.T);
  c.base = p.tree ? c.len : c.len - 1;
  c.lo0 = p.window ? max(0, c.base - p.window + 1) : 0;
  const int n_tiles = (c.len + KT - 1) / KT;
  c.w0 = c.lo0 >= c.len ? n_tiles : c.lo0 / KT;
  c.n_sink = min((min(p.sinks, c.len) + KT - 1) / KT, c.w0);
  c.n_cache = c.n_sink + n_tiles - c.w0;
  c.n = c.m == 0 ? 0 : c.n_cache + (p.tree ? (c.m + KT - 1) / KT : 0);
  return c;
}

// Bits i of a 32-key word at position pos with pos + i < x.
__device__ __forceinline__ uint32_t bits_below(int x, int pos) {
  const int n = min(max(x - pos, 0), 32);
  return n == 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t* r) {
  if constexpr (N == 16) tmem_ld16(a, r);
  else if constexpr (N == 32) tmem_ld32(a, r);
  else if constexpr (N == 64) tmem_ld64(a, r);
  else tmem_ld128(a, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t* r) {
  if constexpr (N == 8) tmem_st8(a, r);
  else if constexpr (N == 16) tmem_st16(a, r);
  else if constexpr (N == 32) tmem_st32(a, r);
  else {
    tmem_st32(a, r);
    tmem_st32(a + 32, r + 32);
  }
}

struct RowState {
  float m, l;
  bool ok;
};

// The softmax of one lane's row over NC keys of each tile (from key col0 of the
// tile on).
template <int D, int NC>
__device__ __forceinline__ RowState cache_softmax(const CacheAttnParams& p, const CacheList& cl, CacheShared* sh,
                                                  uint8_t* sV, uint32_t lane_base, int first, int n, int col0,
                                                  int t_r, const uint32_t* anc, int depth) {
  using C = CacheCfg<D>;
  constexpr int KT = C::KT;
  volatile int* abort = &sh->abort;
  const float sl2 = p.scale_log2;
  const uint32_t s_base = lane_base + C::kS + col0, p_base = lane_base + C::kP + col0 / 2, o_base = lane_base + C::kO;
  // rows of deeper tokens start their window later
  const int lo_r = p.window ? cl.base + depth - p.window + 1 : 0;
  const int lo_last = p.window ? cl.base + cl.m - p.window : 0;
  if (NC < KT) {
    // P of the other repeats' keys stays 0
    uint32_t z[8] = {};
    for (int c = 0; c < KT / 2; c += 8) tmem_st8(lane_base + C::kP + c, z);
  }
  RowState st{-INFINITY, 0.f, true};
  for (int j = 0; j < n && st.ok; ++j) {
    const int i = first + j;
    const bool in_tree = i >= cl.n_cache;
    const int kb = cl.row<KT>(i);
    st.ok = mbar_wait(&sh->s_full, j & 1, abort, p.err, kErrTimeoutCacheAttn);
    tc_fence_after();
    uint32_t s[NC];
    tmem_ld<NC>(s_base, s);
    tc_fence_before();
    mbar_arrive(&sh->s_free);      // S(j) is in registers
    const bool border =
        in_tree || kb + KT > cl.len || (p.window && kb < lo_last && kb + KT > p.sinks);
    if (border) {
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += 32) {
        const int pos = kb + col0 + c0;
        uint32_t vis;
        if (in_tree) {
          vis = anc[pos >> 5];
          if (NC == 16) vis >>= pos & 31;
        } else {
          vis = bits_below(cl.len, pos);
          if (p.window) vis &= ~bits_below(lo_r, pos) | bits_below(p.sinks, pos);
        }
#pragma unroll
        for (int c = 0; c < (NC < 32 ? NC : 32); ++c)
          if (!((vis >> c) & 1u)) s[c0 + c] = __float_as_uint(-INFINITY);
      }
    }
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < NC / 2; ++c)
      m4[c & 3] = fmax3(m4[c & 3], __uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
    const float m_new = fmaxf(st.m, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2);
    // O is rescaled only when some row's max grew by more than 2^8 (l and O
    // share the stale max, so the result is exact)
    bool rescale = false;
    float alpha = 1.f;
    if (j == 0) {
      st.m = m_new;
    } else {
      const bool need = m_new > st.m + kCacheRescaleLog2;
      rescale = __any_sync(0xffffffffu, need);
      if (need) {
        alpha = ex2(st.m - m_new);
        st.l *= alpha;
        st.m = m_new;
      }
    }
    const float neg_m = st.m == -INFINITY ? 0.f : -st.m;     // nothing seen yet: every exponential is 0
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t pk[NC / 2];
#pragma unroll
    for (int c = 0; c < NC / 2; ++c) {
      const float p0 = ex2(fmaf(__uint_as_float(s[2 * c]), sl2, neg_m));
      const float p1 = ex2(fmaf(__uint_as_float(s[2 * c + 1]), sl2, neg_m));
      sum[(c & 1) * 2] += p0;
      sum[(c & 1) * 2 + 1] += p1;
      pk[c] = pack_bf16x2(p0, p1);
    }
    st.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if (j > 0) {
      // P(j-1) V must be done before P is overwritten and O rescaled
      st.ok = mbar_wait(&sh->pv_done, (j - 1) & 1, abort, p.err, kErrTimeoutCacheAttn) && st.ok;
      tc_fence_after();
      if (rescale) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(o_base + c0, o);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tmem_st32(o_base + c0, o);
        }
      }
    }
    tmem_st<NC / 2>(p_base, pk);
    // V rows of keys that no row sees
    const bool dead_keys = in_tree ? kb + KT > cl.m
                                   : kb + KT > cl.len || (p.window && kb < cl.lo0 && kb + KT > p.sinks);
    if (dead_keys) {
      st.ok = mbar_wait(&sh->v_full[j % kCacheST], (j / kCacheST) & 1, abort, p.err, kErrTimeoutCacheAttn) && st.ok;
      const int r = threadIdx.x, pos = kb + r;
      if (r < KT && (in_tree ? pos >= cl.m : pos >= cl.len || (pos < cl.lo0 && pos >= p.sinks))) {
        uint8_t* row = sV + (j % kCacheST) * C::KVBytes + r * 128;
#pragma unroll
        for (int bx = 0; bx < C::NB; ++bx)
#pragma unroll
          for (int q = 0; q < 8; ++q) st_shared_v4(row + bx * C::KBox + q * 16, 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&sh->p_full);
  }
  st.ok = mbar_wait(&sh->pv_done, (n - 1) & 1, abort, p.err, kErrTimeoutCacheAttn) && st.ok;
  tc_fence_after();
  return st;
}

// Where packed row r of group (b, g) lives: token-major, the k routed rows,
// then the shared head's when the group carries it (kr = k + 1).
template <typename T>
__device__ __forceinline__ T* row_ptr(T* routed, T* shared, const CacheAttnParams& p, int bg, int r, int kr, int D) {
  const int t = r / kr, j = r % kr;
  return j < p.k ? routed + ((size_t)((size_t)bg * p.T + t) * p.k + j) * D
                 : shared + ((size_t)(bg / p.G) * p.T + t) * D;
}

template <int D>
__global__ void __launch_bounds__(kCacheThreads, 2)
attn_cache_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                  const __grid_constant__ CUtensorMap mapKt, const __grid_constant__ CUtensorMap mapVt,
                  CacheAttnParams p) {
  using C = CacheCfg<D>;
  constexpr int KT = C::KT, ST = kCacheST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::QBytes;
  uint8_t* sV = sK + ST * C::KVBytes;
  CacheShared* sh = reinterpret_cast<CacheShared*>(sV + ST * C::KVBytes);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int share = blockIdx.x % p.n_split;
  const int qt = blockIdx.x / p.n_split % p.n_qt;
  const int bg = blockIdx.x / p.n_split / p.n_qt;
  const int b = bg / p.G, g = bg % p.G;
  const int kr = p.k + (p.n_shared && g == p.sg ? 1 : 0);
  const int row0 = qt * kRowsQ;
  const int n_rows = min(kRowsQ, p.T * kr - row0);
  if (n_rows <= 0) return;       // only the shared head's group has this query tile
  const int rep = n_rows <= 32 ? 4 : n_rows <= 64 ? 2 : 1;
  const int lanes_rep = kRowsQ / rep;

  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0 && blockIdx.x % (p.n_split * p.n_qt) == 0 && g == 0 && p.err) {
    const int n = p.cache_len[b];
    if (n < (p.tree ? 0 : 1) || n > p.L_max) atomicCAS(p.err, 0u, (unsigned)kErrDecodeCacheLen);
    if (p.tree && p.tree_len && (p.tree_len[b] < 0 || p.tree_len[b] > p.T))
      atomicCAS(p.err, 0u, (unsigned)kErrTreeArgs);
  }
  const CacheList cl = cache_list<KT>(p, b);
  const int first = (int)((long long)cl.n * share / p.n_split);
  const int n = row0 / kr < cl.m ? (int)((long long)cl.n * (share + 1) / p.n_split) - first : 0;

  const size_t item = blockIdx.x;
  float* part_o = p.part + item * p.rows_cap * D;
  float* part_ml = p.part + (size_t)gridDim.x * p.rows_cap * D + item * p.rows_cap * 2;
  if (n == 0) {
    if (p.n_split == 1) {
      for (int e = tid; e < n_rows * (D / 8); e += kCacheThreads)
        reinterpret_cast<uint4*>(row_ptr(p.o_routed, p.o_sh, p, bg, row0 + e / (D / 8), kr, D))[e % (D / 8)] =
            make_uint4(0, 0, 0, 0);
    } else {
      for (int e = tid; e < n_rows; e += kCacheThreads) {
        part_ml[2 * e] = -INFINITY;
        part_ml[2 * e + 1] = 0.f;
      }
    }
    return;
  }

  auto load_k = [&](int j) {
    const int s = j % ST, i = first + j;
    const CUtensorMap* map = i < cl.n_cache ? &mapK : &mapKt;
    mbar_arrive_expect_tx(&sh->k_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sK + s * C::KVBytes + bx * C::KBox, map, &sh->k_full[s], bx * 64, cl.row<KT>(i), bg);
  };
  auto load_v = [&](int j) {
    const int s = j % ST, i = first + j;
    const CUtensorMap* map = i < cl.n_cache ? &mapV : &mapVt;
    mbar_arrive_expect_tx(&sh->v_full[s], C::KVBytes);
    for (int bx = 0; bx < C::NB; ++bx)
      tma_load_3d(sV + s * C::KVBytes + bx * C::KBox, map, &sh->v_full[s], bx * 64, cl.row<KT>(i), bg);
  };
  if (warp == 4 && lane == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sh->k_full[s], 1);
      mbar_init(&sh->k_empty[s], 1);
      mbar_init(&sh->v_full[s], 1);
      mbar_init(&sh->v_empty[s], 1);
    }
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->s_free, 128);
    mbar_init(&sh->p_full, 128);
    mbar_init(&sh->pv_done, 1);
    sh->abort = 0;
    fence_mbar_init();
    for (int j = 0; j < ST && j < n; ++j) {
      load_k(j);
      load_v(j);
    }
  }
  if (warp == 5) tmem_alloc(&sh->tmem_base, 256);
  // Q rows, repeated `rep` times, into the 128-byte swizzled layout
  for (int e = tid; e < kRowsQ * (D / 8); e += kCacheThreads) {
    const int L = e / (D / 8), c = e % (D / 8), r = L % lanes_rep;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < n_rows) v = reinterpret_cast<const uint4*>(row_ptr(p.q_routed, p.q_sh, p, bg, row0 + r, kr, D))[c];
    st_shared_v4(sQ + (c >> 3) * C::QBox + L * 128 + (((c & 7) ^ (L & 7)) << 4), v.x, v.y, v.z, v.w);
  }
  // ancestors and depths of the drafted tokens by pointer doubling: after round
  // r a token's bits cover 2^(r+1) - 1 levels above it
  int cur = 0;
  if (p.tree) {
    if (tid < p.T) {
      int up = tid < cl.m ? p.parent[(size_t)b * p.T + tid] : -1;
      if (up < -1 || up >= tid) {
        if (p.err) atomicCAS(p.err, 0u, (unsigned)kErrTreeArgs);
        up = -1;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w)
        sh->anc[0][tid][w] = ((tid >> 5) == w ? 1u << (tid & 31) : 0u) |
                             (up >= 0 && (up >> 5) == w ? 1u << (up & 31) : 0u);
      sh->up[0][tid] = up;
      sh->depth[0][tid] = up >= 0 ? 1 : 0;
    }
    for (int span = 1; span < p.T; span *= 2) {
      __syncthreads();
      if (tid < p.T) {
        const int up = sh->up[cur][tid];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          sh->anc[cur ^ 1][tid][w] = sh->anc[cur][tid][w] | (up >= 0 ? sh->anc[cur][up][w] : 0u);
        sh->depth[cur ^ 1][tid] = sh->depth[cur][tid] + (up >= 0 ? sh->depth[cur][up] : 0);
        sh->up[cur ^ 1][tid] = up >= 0 ? sh->up[cur][up] : -1;
      }
      cur ^= 1;
    }
    __syncthreads();
    if (p.window && p.window < p.T && tid < p.T) {
      // ancestors that the window has left behind
      for (int a = 0; a < tid; ++a)
        if (sh->depth[cur][tid] - sh->depth[cur][a] >= p.window && cl.base + sh->depth[cur][a] >= p.sinks)
          sh->anc[cur][tid][a >> 5] &= ~(1u << (a & 31));
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp == 4) {
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRowsQ, KT, false, false);
      const uint32_t q0 = smem_u32(sQ);
      bool ok = true;
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % ST;
        if (j > 0) ok = mbar_wait(&sh->s_free, (j - 1) & 1, abort, p.err, kErrTimeoutCacheAttn);
        ok = ok && mbar_wait(&sh->k_full[s], (j / ST) & 1, abort, p.err, kErrTimeoutCacheAttn);
        if (!ok) break;
        tc_fence_after();
        const uint32_t k0 = smem_u32(sK + s * C::KVBytes);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_ss(tmem + C::kS, sdesc_sw128(q0 + (ks >> 2) * C::QBox + (ks & 3) * 32, 16, 1024),
                  sdesc_sw128(k0 + (ks >> 2) * C::KBox + (ks & 3) * 32, 16, 1024), idesc_s, ks > 0);
        umma_commit(&sh->s_full);
        umma_commit(&sh->k_empty[s]);
        if (j + ST < n) {
          ok = mbar_wait(&sh->k_empty[s], (j / ST) & 1, abort, p.err, kErrTimeoutCacheAttn);
          if (!ok) break;
          load_k(j + ST);
        }
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc_o = idesc_bf16_f32(kRowsQ, D, false, true);
      for (int j = 0; j < n; ++j) {
        const int s = j % ST;
        if (!mbar_wait(&sh->p_full, j & 1, abort, p.err, kErrTimeoutCacheAttn)) break;
        if (!mbar_wait(&sh->v_full[s], (j / ST) & 1, abort, p.err, kErrTimeoutCacheAttn)) break;
        tc_fence_after();
        const uint32_t v0 = smem_u32(sV + s * C::KVBytes);
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks)
          umma_ts(tmem + C::kO, tmem + C::kP + ks * 8, sdesc_sw128(v0 + ks * 2048, C::KBox, 1024), idesc_o,
                  (j > 0 || ks > 0));
        umma_commit(&sh->pv_done);
        umma_commit(&sh->v_empty[s]);
        if (j + ST < n) {
          if (!mbar_wait(&sh->v_empty[s], (j / ST) & 1, abort, p.err, kErrTimeoutCacheAttn)) break;
          load_v(j + ST);
        }
      }
    }
  } else {
    // ---------------- softmax: warps 0-3, one lane per (row, repeat)
    const int r = tid % lanes_rep, q = tid / lanes_rep;
    const int t_r = (row0 + r) / kr;
    const bool live = r < n_rows && t_r < cl.m;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int depth = p.tree && live ? sh->depth[cur][t_r] : 0;
    const uint32_t* anc = sh->anc[cur][live ? t_r : 0];
    RowState st;
    if (rep == 4)
      st = cache_softmax<D, KT / 4>(p, cl, sh, sV, lane_base, first, n, q * (KT / 4), t_r, anc, depth);
    else if (rep == 2)
      st = cache_softmax<D, KT / 2>(p, cl, sh, sV, lane_base, first, n, q * (KT / 2), t_r, anc, depth);
    else
      st = cache_softmax<D, KT>(p, cl, sh, sV, lane_base, first, n, 0, t_r, anc, depth);
    // ---------------- epilogue: join the repeats through shared memory (the
    // operand tiles are no longer read)
    float* sO = reinterpret_cast<float*>(smem);
    sh->m[tid] = live ? st.m : -INFINITY;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    float M = -INFINITY;
    for (int i = 0; i < rep; ++i) M = fmaxf(M, sh->m[r + i * lanes_rep]);
    const float f = live && st.m > -INFINITY ? ex2(st.m - M) : 0.f;
    sh->l[tid] = f > 0.f ? st.l * f : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      tmem_ld32(lane_base + C::kO + c0, o);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (f > 0.f)
          v = make_float4(__uint_as_float(o[4 * c]) * f, __uint_as_float(o[4 * c + 1]) * f,
                          __uint_as_float(o[4 * c + 2]) * f, __uint_as_float(o[4 * c + 3]) * f);
        reinterpret_cast<float4*>(sO + tid * C::OPitch + c0)[c] = v;
      }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const bool aborted = *abort != 0;
    for (int e = tid; e < n_rows * (D / 8) && !aborted; e += 128) {
      const int er = e / (D / 8), c8 = e % (D / 8);
      float a[8] = {}, Ls = 0.f, Ms = -INFINITY;
      for (int i = 0; i < rep; ++i) {
        const int L = er + i * lanes_rep;
        const float4 x = reinterpret_cast<const float4*>(sO + L * C::OPitch)[c8 * 2];
        const float4 y = reinterpret_cast<const float4*>(sO + L * C::OPitch)[c8 * 2 + 1];
        a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
        a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
        Ls += sh->l[L];
        Ms = fmaxf(Ms, sh->m[L]);
      }
      if (p.n_split == 1) {
        const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
        reinterpret_cast<uint4*>(row_ptr(p.o_routed, p.o_sh, p, bg, row0 + er, kr, D))[c8] =
            make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                       pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
      } else {
        float4* d4 = reinterpret_cast<float4*>(part_o + er * D + c8 * 8);
        d4[0] = make_float4(a[0], a[1], a[2], a[3]);
        d4[1] = make_float4(a[4], a[5], a[6], a[7]);
        if (c8 == 0) {
          part_ml[2 * er] = Ms;
          part_ml[2 * er + 1] = Ls;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  drain_after_abort(abort);
}

// Joins the shares of every row: o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
// Eight columns per thread; rows that saw nothing get 0.
template <int D>
__global__ void __launch_bounds__(256) attn_cache_merge_kernel(CacheAttnParams p, long long n_items) {
  pdl_launch_dependents();
  pdl_wait();
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const int c8 = (int)(e % (D / 8));
  const int r = (int)(e / (D / 8) % p.rows_cap);
  const long long tile = e / (D / 8) / p.rows_cap;      // (b, g, query tile)
  if (tile * p.n_split >= n_items) return;
  const int bg = (int)(tile / p.n_qt), row0 = (int)(tile % p.n_qt) * kRowsQ;
  const int kr = p.k + (p.n_shared && bg % p.G == p.sg ? 1 : 0);
  if (row0 + r >= p.T * kr) return;
  const float* ml = p.part + (size_t)n_items * p.rows_cap * D + ((size_t)tile * p.n_split * p.rows_cap + r) * 2;
  const float* po = p.part + ((size_t)tile * p.n_split * p.rows_cap + r) * D + c8 * 8;
  float M = -INFINITY;
  for (int c = 0; c < p.n_split; ++c) M = fmaxf(M, ml[(size_t)c * p.rows_cap * 2]);
  float a[8] = {}, Ls = 0.f;
  for (int c = 0; c < p.n_split; ++c) {
    const float mc = ml[(size_t)c * p.rows_cap * 2];
    if (mc == -INFINITY) continue;         // nothing seen: its O was not written
    const float f = ex2(mc - M);
    const float4 x = reinterpret_cast<const float4*>(po + (size_t)c * p.rows_cap * D)[0];
    const float4 y = reinterpret_cast<const float4*>(po + (size_t)c * p.rows_cap * D)[1];
    Ls = fmaf(ml[(size_t)c * p.rows_cap * 2 + 1], f, Ls);
    a[0] = fmaf(x.x, f, a[0]), a[1] = fmaf(x.y, f, a[1]), a[2] = fmaf(x.z, f, a[2]), a[3] = fmaf(x.w, f, a[3]);
    a[4] = fmaf(y.x, f, a[4]), a[5] = fmaf(y.y, f, a[5]), a[6] = fmaf(y.z, f, a[6]), a[7] = fmaf(y.w, f, a[7]);
  }
  const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
  reinterpret_cast<uint4*>(row_ptr(p.o_routed, p.o_sh, p, bg, row0 + r, kr, D))[c8] =
      make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                 pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
}

// Accepted drafted rows to the end of the cache: one CTA per sequence, so that
// new_len may be cache_len itself (the CTA has read it before it writes).
__global__ void __launch_bounds__(512) cache_commit_kernel(CommitParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x;
  int len = p.cache_len[b], n = p.n_accept[b];
  bool bad = false;
  if (len < 0 || len > p.L_max) bad = true, len = min(max(len, 0), p.L_max);
  if (n < 0 || n > p.T) bad = true, n = min(max(n, 0), p.T);
  if (n > p.L_max - len) bad = true, n = p.L_max - len;
  const int c8n = p.d / 8;
  const uint4* src[2] = {reinterpret_cast<const uint4*>(p.Kt), reinterpret_cast<const uint4*>(p.Vt)};
  uint4* dst[2] = {reinterpret_cast<uint4*>(p.Kc), reinterpret_cast<uint4*>(p.Vc)};
  for (int e = threadIdx.x; e < n * p.G * c8n; e += 512) {
    const int c8 = e % c8n, i = e / c8n % n, g = e / c8n / n;
    const int node = p.path[(size_t)b * p.T + i];
    if (node < 0 || node >= p.T) {       // no such drafted token: its cache row stays as it was
      bad = true;
      continue;
    }
    const size_t from = (((size_t)b * p.G + g) * p.T + node) * c8n + c8;
    const size_t to = (((size_t)b * p.G + g) * p.L_max + len + i) * c8n + c8;
    dst[0][to] = src[0][from];
    dst[1][to] = src[1][from];
  }
  if (bad && p.err) atomicCAS(p.err, 0u, (unsigned)kErrCommitArgs);
  __syncthreads();
  if (threadIdx.x == 0) p.new_len[b] = len + n;
}

// Key tiles a sequence can have at most (window 0: the whole cache).
long long max_tiles(int L_max, int T, bool tree, int window, int sinks, int KT) {
  long long cache = ((long long)L_max + KT - 1) / KT;
  if (window) {
    const long long w = ((long long)window + KT - 2) / KT + 1 + ((long long)sinks + KT - 1) / KT;
    if (w < cache) cache = w;
  }
  return cache + (tree ? (T + KT - 1) / KT : 0);
}

}  // namespace

void cache_attn_plan(int B, int T, int G, int k, int n_shared, int d, int L_max, bool tree, int window, int sinks,
                     CacheAttnPlan* P) {
  const int KT = d == 64 ? 128 : 64;
  const int rows = T * (k + n_shared);
  P->n_qt = (rows + kRowsQ - 1) / kRowsQ;
  P->rows_cap = rows < kRowsQ ? rows : kRowsQ;
  // Shares per query tile: the fewest that come within a twentieth of the
  // shortest time of ceil(items * shares / slots) waves of (tiles per share +
  // start-up) each; 296 slots are two CTAs on each of 148 SMs, and a CTA's
  // start-up and end cost about as much as four tiles.
  const long long items = (long long)B * G * P->n_qt, nt = max_tiles(L_max, T, tree, window, sinks, KT);
  const long long slots = 296, startup = 4;
  long long best = 0;
  int cap = (int)(nt < 32 ? nt : 32);
  auto cost = [&](int n) { return (items * n + slots - 1) / slots * ((nt + n - 1) / n + startup); };
  for (int n = 1; n <= cap; ++n)
    if (n == 1 || cost(n) < best) best = cost(n);
  P->n_split = 1;
  for (int n = 1; n <= cap; ++n)
    if (cost(n) * 20 <= best * 21) {
      P->n_split = n;
      break;
    }
  P->items = items * P->n_split;
  P->bytes = P->n_split == 1 ? 0 : (size_t)P->items * P->rows_cap * (d + 2) * sizeof(float);
}

template <int D>
static cudaError_t launch_cache(const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mKt,
                                const CUtensorMap& mVt, const CacheAttnParams& p, long long items,
                                cudaStream_t stream) {
  auto kern = attn_cache_kernel<D>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), cache_smem<D>());
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3((unsigned)items), dim3(kCacheThreads), cache_smem<D>(), stream, 1, mK, mV, mKt, mVt, p);
  if (e != cudaSuccess || p.n_split == 1) return e;
  const long long threads = items / p.n_split * p.rows_cap * (D / 8);
  return launch_kernel(attn_cache_merge_kernel<D>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, 1, p,
                       items);
}

cudaError_t launch_attn_cache(const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mKt,
                              const CUtensorMap& mVt, const CacheAttnParams& p, int d, long long items,
                              cudaStream_t stream) {
  if (items > 0x7FFFFFFFll) return cudaErrorNotSupported;
  return d == 64 ? launch_cache<64>(mK, mV, mKt, mVt, p, items, stream)
                 : launch_cache<128>(mK, mV, mKt, mVt, p, items, stream);
}

cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t stream) {
  return launch_kernel(cache_commit_kernel, dim3(p.B), dim3(512), 0, stream, 1, p);
}

}  // namespace gqe
