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
// is the shared head's, are packed into 128-row query tiles; each query tile
// reads the group's key tiles once (from L2 after the first, where a group has
// more than 128 rows).  Work item: one query tile of one (b, g) and a share of its
// key list.  The CTAs of one query tile's shares form a cluster:
// each leaves its rows' softmax state (max, sum, unnormalised O, fp32) in its
// own shared memory, and after a cluster barrier the CTAs divide the rows among
// them and join the states over distributed shared memory.
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
//
// Bound by HBM where there are many keys: 64 sequences under a 4096-token window
// (d = 64, 8 groups) 87 to 90 us, 0.92 to 0.96 of the measured copy bandwidth; 64
// trees of 32 tokens over 32768-token caches 625 to 675 us, 0.99 and more.  Few keys:
// by latency, start 3 us, about 1 us a key tile, join 2-3 us (one tree of 8 tokens,
// 4096 rows: 10.1 us).  GPU times in a captured graph, by box.
#include "attn.cuh"
#include "launch.cuh"

namespace gqe {

namespace {

constexpr int kRowsQ = 128;       // query rows per tile
constexpr int kCacheThreads = 192;
constexpr float kCacheRescaleLog2 = 8.0f;

template <int D>
struct CacheCfg {
  static constexpr int NB = D / 64;
  static constexpr int KT = D == 64 ? 128 : 64;          // keys per tile
  static constexpr int KST = D == 64 ? 3 : 2;            // K and V ring depths
  static constexpr int VST = 2;
  static constexpr int QBox = kRowsQ * 128;              // 128 rows x 64 bf16
  static constexpr int KBox = KT * 128;
  static constexpr int QBytes = NB * QBox;
  static constexpr int KVBytes = NB * KBox;
  static constexpr uint32_t kS = 0, kP = KT, kO = D == 64 ? 192 : 128;
  static constexpr int OPitch = D + 4;                   // floats per staged O row
};

struct __align__(16) CacheShared {
  uint4 anc[2][kMaxTree];            // ancestor bits (double-buffered while they are built)
  int up[2][kMaxTree];               // pointer doubling: 2^r levels up, -1 past the root
  int depth[2][kMaxTree];
  float m[kRowsQ], l[kRowsQ];        // per lane
  float2 row_ml[kRowsQ];             // per row, its repeats joined
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full, s_free, p_full, pv_done;
  uint32_t tmem_base;
  int abort;
};

template <int D>
constexpr size_t cache_smem() {
  using C = CacheCfg<D>;
  return 1024 + C::QBytes + (C::KST + C::VST) * C::KVBytes + sizeof(CacheShared);
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

struct RowState {
  float m, l;
  bool ok;
};

// The softmax of one lane's row over NC keys of each tile (from key col0 of the
// tile on).
template <int D, int NC>
__device__ __forceinline__ RowState cache_softmax(const CacheAttnParams& p, const CacheList& cl, CacheShared* sh,
                                                  uint8_t* sV, uint32_t lane_base, int first, int n, int col0,
                                                  const uint32_t* anc, int depth) {
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
    st.ok = mbar_wait_short(&sh->s_full, j & 1, abort);
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
    const unsigned long long sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg_m, neg_m);
    unsigned long long sum2[2] = {0ull, 0ull};
    uint32_t pk[NC / 2];
#pragma unroll
    for (int c = 0; c < NC / 2; ++c) {
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, negm2), x0, x1);
      x0 = ex2(x0);
      x1 = ex2(x1);
      sum2[c & 1] = f2_add(sum2[c & 1], f2_pack(x0, x1));
      pk[c] = pack_bf16x2(x0, x1);
    }
    {
      float a0, a1, b0, b1;
      f2_unpack(sum2[0], a0, a1);
      f2_unpack(sum2[1], b0, b1);
      st.l += (a0 + a1) + (b0 + b1);
    }
    if (j > 0) {
      // P(j-1) V must be done before P is overwritten and O rescaled
      st.ok = mbar_wait_short(&sh->pv_done, (j - 1) & 1, abort) && st.ok;
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
      st.ok = mbar_wait_short(&sh->v_full[j % C::VST], (j / C::VST) & 1, abort) && st.ok;
      const int r = threadIdx.x, pos = kb + r;
      if (r < KT && (in_tree ? pos >= cl.m : pos >= cl.len || (pos < cl.lo0 && pos >= p.sinks))) {
        uint8_t* row = sV + (j % C::VST) * C::KVBytes + r * 128;
#pragma unroll 1
        for (int q = 0; q < C::NB * 8; ++q) st_shared_v4(row + (q >> 3) * C::KBox + (q & 7) * 16, 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&sh->p_full);
  }
  st.ok = mbar_wait_short(&sh->pv_done, (n - 1) & 1, abort) && st.ok;
  tc_fence_after();
  return st;
}

// The packed rows of group (b, g): token-major, the k routed rows, then the
// shared head's when the group carries it (kr = k + 1).
struct RowMap {
  int k, kr;
  unsigned inv;        // ceil(2^20 / kr): r / kr is exact for r < 1152 and kr <= 9
  size_t routed, shared;    // first element of the group's routed rows, of the sequence's shared rows
  __device__ __forceinline__ RowMap(const CacheAttnParams& p, int bg, int b, int kr_, int D)
      : k(p.k), kr(kr_), inv(((1u << 20) + kr_ - 1) / kr_), routed((size_t)bg * p.T * p.k * D),
        shared((size_t)b * p.T * D) {}
  __device__ __forceinline__ int token(int r) const { return (int)((r * inv) >> 20); }
  template <typename T>
  __device__ __forceinline__ T* at(T* q_routed, T* q_sh, int r, int D) const {
    const int t = token(r), j = r - t * kr;
    return j < k ? q_routed + routed + (size_t)(t * k + j) * D : q_sh + shared + (size_t)t * D;
  }
};

// Ancestor bits and depths of the drafted tokens by pointer doubling, on the
// 128 threads of the softmax warps: a token starts with itself and one level, and
// after round r = 0, 1, .. its bits cover the 2^(r+1) levels above it.  up: thread
// i's parent[i].  Returns the buffer that holds the result.
__device__ __forceinline__ int build_tree(const CacheAttnParams& p, const CacheList& cl, CacheShared* sh, int up) {
  const int i = threadIdx.x;
  if (up < -1 || up >= i) {
    if (p.err) atomicCAS(p.err, 0u, (unsigned)kErrTreeArgs);
    up = -1;
  }
  uint32_t own[4];
#pragma unroll
  for (int w = 0; w < 4; ++w)
    own[w] = ((i >> 5) == w ? 1u << (i & 31) : 0u) | (up >= 0 && (up >> 5) == w ? 1u << (up & 31) : 0u);
  uint4 anc = make_uint4(own[0], own[1], own[2], own[3]);
  int depth = up >= 0 ? 1 : 0, cur = 0;
  for (int span = 1; span < p.T; span *= 2) {
    if (i < p.T) {
      sh->anc[cur][i] = anc;
      sh->depth[cur][i] = depth;
      sh->up[cur][i] = up;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (up >= 0) {
      const uint4 a = sh->anc[cur][up];
      anc.x |= a.x, anc.y |= a.y, anc.z |= a.z, anc.w |= a.w;
      depth += sh->depth[cur][up];
      up = sh->up[cur][up];
    }
    cur ^= 1;
  }
  if (i < p.T) {
    sh->anc[cur][i] = anc;
    sh->depth[cur][i] = depth;
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  if (p.window && p.window < p.T && i < p.T) {
    // ancestors that the window has left behind
    uint32_t* bits = reinterpret_cast<uint32_t*>(&sh->anc[cur][i]);
    for (int a = 0; a < i; ++a)
      if (depth - sh->depth[cur][a] >= p.window && cl.base + sh->depth[cur][a] >= p.sinks)
        bits[a >> 5] &= ~(1u << (a & 31));
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  return cur;
}

// Joins the shares of a query tile's rows and writes them:
// o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the CTAs c of the
// cluster (one CTA: no cluster), four columns per thread; rows that saw
// nothing get 0.  Every thread of the CTA calls it; a CTA leaves only when the
// others have read its shared memory.
template <int D>
__device__ __forceinline__ void join_shares(const CacheAttnParams& p, CacheShared* sh, const uint8_t* smem,
                                            const RowMap& rows, int row0, int n_rows) {
  constexpr int OPitch = CacheCfg<D>::OPitch;
  const float* sO = reinterpret_cast<const float*>(smem);
  const int share = blockIdx.x % p.n_split;
  if (p.n_split > 1) {
    __syncwarp();
    cluster_sync();
  }
  const bool ok = *static_cast<volatile int*>(&sh->abort) == 0;
  // A warp takes 32/S four-column pieces at a time, each by S lanes (a power of
  // two) that take every S-th share, at most kJoin each.  Lanes side by side read
  // one CTA's memory side by side.  63 tokens' 252 rows in three shares (d = 128)
  // 25.3 us a call, with two shares a lane 28.6, one 36.9, eight 26.1; two pieces
  // at once 25.6.
  constexpr int kJoin = 4;
  int S = 1;
  while (S * kJoin < p.n_split) S *= 2;
  const int lane = threadIdx.x & 31, side = 32 / S, sub = lane / side;
  const int n_units = n_rows * (D / 4), warps = p.n_split * (kCacheThreads / 32);
  for (int u0 = (share * (kCacheThreads / 32) + (threadIdx.x >> 5)) * side; u0 < n_units; u0 += warps * side) {
    const int u = u0 + lane % side, er = u / (D / 4), c4 = u % (D / 4);
    float2 ml[kJoin];
    float4 x[kJoin];
#pragma unroll
    for (int h = 0; h < kJoin; ++h) {
      const int c = sub + h * S;
      ml[h] = make_float2(-INFINITY, 0.f);
      x[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ok && u < n_units && c < p.n_split) {
        // (one CTA reads itself through the same instructions: rank 0 of 1)
        ml[h] = ld_cluster_f32x2(cluster_map(smem_u32(&sh->row_ml[er]), c));
        x[h] = ld_cluster_f32x4(cluster_map(smem_u32(sO + er * OPitch + c4 * 4), c));
      }
    }
    float M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int h = 0; h < kJoin; ++h) M = fmaxf(M, ml[h].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int o = side; o < 32; o *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int h = 0; h < kJoin; ++h) {
      if (ml[h].y != 0.f) {              // else the share saw nothing and its O was not written
        const float f = ex2(ml[h].x - M);
        Ls = fmaf(ml[h].y, f, Ls);
        a.x = fmaf(x[h].x, f, a.x), a.y = fmaf(x[h].y, f, a.y);
        a.z = fmaf(x[h].z, f, a.z), a.w = fmaf(x[h].w, f, a.w);
      }
    }
    for (int o = side; o < 32; o *= 2) {
      Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
      a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;        // a NaN sum stays one
    if (ok && u < n_units && sub == 0)
      reinterpret_cast<uint2*>(rows.at(p.o_routed, p.o_sh, row0 + er, D))[c4] =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
  if (p.n_split > 1) {
    __syncwarp();
    cluster_sync_relaxed();
  }
}

template <int D>
__global__ void __launch_bounds__(kCacheThreads, 2)
attn_cache_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                  const __grid_constant__ CUtensorMap mapKt, const __grid_constant__ CUtensorMap mapVt,
                  CacheAttnParams p) {
  using C = CacheCfg<D>;
  constexpr int KT = C::KT, KST = C::KST, VST = C::VST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::QBytes;
  uint8_t* sV = sK + KST * C::KVBytes;
  CacheShared* sh = reinterpret_cast<CacheShared*>(sV + VST * C::KVBytes);
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

  pdl_wait();
  if (tid == 0 && blockIdx.x % (p.n_split * p.n_qt) == 0 && g == 0 && p.err) {
    const int n = p.cache_len[b];
    if (n < (p.tree ? 0 : 1) || n > p.L_max) atomicCAS(p.err, 0u, (unsigned)kErrDecodeCacheLen);
    if (p.tree && p.tree_len && (p.tree_len[b] < 0 || p.tree_len[b] > p.T))
      atomicCAS(p.err, 0u, (unsigned)kErrTreeArgs);
  }
  const CacheList cl = cache_list<KT>(p, b);
  const RowMap rows(p, bg, b, kr, D);
  const int first = (int)((long long)cl.n * share / p.n_split);
  const int n = rows.token(row0) < cl.m ? (int)((long long)cl.n * (share + 1) / p.n_split) - first : 0;

  if (n > 0) {
    auto load_k = [&](int j) {
      const int s = j % KST, i = first + j;
      const CUtensorMap* map = i < cl.n_cache ? &mapK : &mapKt;
      mbar_arrive_expect_tx(&sh->k_full[s], C::KVBytes);
      for (int bx = 0; bx < C::NB; ++bx)
        tma_load_3d(sK + s * C::KVBytes + bx * C::KBox, map, &sh->k_full[s], bx * 64, cl.row<KT>(i), bg);
    };
    auto load_v = [&](int j) {
      const int s = j % VST, i = first + j;
      const CUtensorMap* map = i < cl.n_cache ? &mapV : &mapVt;
      mbar_arrive_expect_tx(&sh->v_full[s], C::KVBytes);
      for (int bx = 0; bx < C::NB; ++bx)
        tma_load_3d(sV + s * C::KVBytes + bx * C::KBox, map, &sh->v_full[s], bx * 64, cl.row<KT>(i), bg);
    };
    if (warp == 4 && lane == 0) {
      for (int s = 0; s < KST; ++s) {
        mbar_init(&sh->k_full[s], 1);
        mbar_init(&sh->k_empty[s], 1);
      }
      for (int s = 0; s < VST; ++s) {
        mbar_init(&sh->v_full[s], 1);
        mbar_init(&sh->v_empty[s], 1);
      }
      mbar_init(&sh->s_full, 1);
      mbar_init(&sh->s_free, 128);
      mbar_init(&sh->p_full, 128);
      mbar_init(&sh->pv_done, 1);
      sh->abort = 0;
      fence_mbar_init();
      for (int j = 0; j < KST && j < n; ++j) {
        load_k(j);
        if (j < VST) load_v(j);
      }
    }
    if (warp == 5) tmem_alloc(&sh->tmem_base, 256);
    const int up = p.tree && tid < cl.m ? p.parent[(size_t)b * p.T + tid] : -1;
    // Q rows, repeated `rep` times, into the 128-byte swizzled layout (every load
    // in flight before the first store: one trip to memory)
    {
      constexpr int NL = (kRowsQ * (D / 8) + kCacheThreads - 1) / kCacheThreads;
      uint4 v[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = tid + i * kCacheThreads, r = e / (D / 8);
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < n_rows) v[i] = reinterpret_cast<const uint4*>(rows.at(p.q_routed, p.q_sh, row0 + r, D))[e % (D / 8)];
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = tid + i * kCacheThreads, c = e % (D / 8);
        if (e / (D / 8) < lanes_rep)
          for (int L = e / (D / 8); L < kRowsQ; L += lanes_rep)
            st_shared_v4(sQ + (c >> 3) * C::QBox + L * 128 + (((c & 7) ^ (L & 7)) << 4), v[i].x, v[i].y, v[i].z,
                         v[i].w);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;
    // Behind the allocation: a dependent CTA may start on this SM at the signal, and
    // allocate columns that it keeps while it waits for this grid.
    pdl_launch_dependents();

    if (warp == 4) {
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRowsQ, KT, false, false);
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      for (int j = 0; j < n; ++j) {
        const int s = j % KST;
        if (j > 0 && !mbar_wait_warp(&sh->s_free, (j - 1) & 1, abort)) break;
        if (!mbar_wait_warp(&sh->k_full[s], (j / KST) & 1, abort)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t dk = sdesc_sw128(smem_u32(sK + s * C::KVBytes), 16, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_ss(tmem + C::kS, sdesc_at(dq, (ks >> 2) * C::QBox + (ks & 3) * 32),
                    sdesc_at(dk, (ks >> 2) * C::KBox + (ks & 3) * 32), idesc_s, ks > 0);
          umma_commit(&sh->s_full);
          umma_commit(&sh->k_empty[s]);
        }
        if (j + KST < n) {
          if (!mbar_wait_warp(&sh->k_empty[s], (j / KST) & 1, abort)) break;
          if (leader) load_k(j + KST);
        }
      }
    } else if (warp == 5) {
      const bool leader = elect_one();
      constexpr uint32_t idesc_o = idesc_bf16_f32(kRowsQ, D, false, true);
      for (int j = 0; j < n; ++j) {
        const int s = j % VST;
        if (!mbar_wait_warp(&sh->p_full, j & 1, abort)) break;
        if (!mbar_wait_warp(&sh->v_full[s], (j / VST) & 1, abort)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t dv = sdesc_sw128(smem_u32(sV + s * C::KVBytes), C::KBox, 1024);
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            umma_ts(tmem + C::kO, tmem + C::kP + ks * 8, sdesc_at(dv, ks * 2048), idesc_o, (j > 0 || ks > 0));
          umma_commit(&sh->pv_done);
          umma_commit(&sh->v_empty[s]);
        }
        if (j + VST < n) {
          if (!mbar_wait_warp(&sh->v_empty[s], (j / VST) & 1, abort)) break;
          if (leader) load_v(j + VST);
        }
      }
    } else {
      // ---------------- softmax: warps 0-3, one lane per (row, repeat)
      const int cur = p.tree ? build_tree(p, cl, sh, up) : 0;
      const int r = tid % lanes_rep, q = tid / lanes_rep;
      const int t_r = rows.token(row0 + r);
      const bool live = r < n_rows && t_r < cl.m;
      const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
      const int depth = p.tree && live ? sh->depth[cur][t_r] : 0;
      const uint32_t* anc = reinterpret_cast<const uint32_t*>(&sh->anc[cur][live ? t_r : 0]);
      RowState st;
      if (rep == 4)
        st = cache_softmax<D, KT / 4>(p, cl, sh, sV, lane_base, first, n, q * (KT / 4), anc, depth);
      else if (rep == 2)
        st = cache_softmax<D, KT / 2>(p, cl, sh, sV, lane_base, first, n, q * (KT / 2), anc, depth);
      else
        st = cache_softmax<D, KT>(p, cl, sh, sV, lane_base, first, n, 0, anc, depth);
      // ---------------- epilogue: join the repeats through shared memory (the
      // operand tiles are no longer read)
      float* sO = reinterpret_cast<float*>(smem);
      sh->m[tid] = live ? st.m : -INFINITY;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      float M = -INFINITY;
      for (int i = 0; i < rep; ++i) M = fmaxf(M, sh->m[r + i * lanes_rep]);
      const bool saw = live && st.l != 0.f;       // (a NaN sum is one too, and reaches the output)
      const float f = saw ? ex2(st.m - M) : 0.f;
      sh->l[tid] = saw ? st.l * f : 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(lane_base + C::kO + c0, o);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (saw)
            v = make_float4(__uint_as_float(o[4 * c]) * f, __uint_as_float(o[4 * c + 1]) * f,
                            __uint_as_float(o[4 * c + 2]) * f, __uint_as_float(o[4 * c + 3]) * f);
          reinterpret_cast<float4*>(sO + tid * C::OPitch + c0)[c] = v;
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // the sum over a row's repeats replaces its first repeat
      for (int e = tid; rep > 1 && e < n_rows * (D / 4); e += 128) {
        const int er = e / (D / 4), c4 = e % (D / 4);
        float4* first_o = reinterpret_cast<float4*>(sO + er * C::OPitch) + c4;
        float4 a = *first_o;
        for (int i = 1; i < rep; ++i) {
          const float4 x = reinterpret_cast<const float4*>(sO + (er + i * lanes_rep) * C::OPitch)[c4];
          a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
        }
        *first_o = a;
      }
      if (tid < n_rows) {
        float Ls = 0.f;
        for (int i = 0; i < rep; ++i) Ls += sh->l[tid + i * lanes_rep];
        sh->row_ml[tid] = make_float2(M, Ls);
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
      drain_after_abort(abort);      // what is in flight lands before another CTA gets the columns
      tc_fence_after();
      tmem_dealloc(tmem, 256);
    }
  } else {
    pdl_launch_dependents();
    // an empty share: its rows saw nothing
    if (tid < n_rows) sh->row_ml[tid] = make_float2(-INFINITY, 0.f);
    if (tid == 0) sh->abort = 0;
    __syncthreads();
  }
  join_shares<D>(p, sh, smem, rows, row0, n_rows);
  report_abort(abort, p.err, kErrTimeoutCacheAttn);
}

// Accepted drafted rows to the end of the cache: one CTA per sequence, so that
// new_len may be cache_len itself (the CTA has read it before it writes).  Bound by
// latency (lengths, path, row, one after the other): 2.0 us for one sequence, 3.5
// us for 64 sequences of 17 rows of 8 groups, of which the bytes are 0.3 us.
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
  // Shares per query tile (the CTAs of a cluster: at most 16), by a model of the
  // time in units of one key tile of a CTA that has its SM to itself (about
  // 1 us): start-up and end 5, a tile 4/3 when two CTAs share an SM, a quarter
  // for each CTA of the cluster's barriers, all of it once per 296 CTAs (two on
  // each of 148 SMs) but at least once.  Measured (us): 64 x 8 items of 33 tiles
  // 95, 109, 121 for 1, 2, 3 shares; 20 items of 17 tiles 12.7, 10.0, 8.8, 10.0
  // for 2, 4, 6, 8; 72 items of 35 tiles 43, 27, 25, 28, 36 for 1, 2, 3, 4, 6; 8
  // items of 33 tiles 16.8, 12.2, 10.4, 10.0 for 2, 4, 6, 8.
  const long long items = (long long)B * G * P->n_qt, nt = max_tiles(L_max, T, tree, window, sinks, KT);
  const int cap = (int)(nt < 16 ? nt : 16);
  double best = 0;
  for (int n = 1; n <= cap; ++n) {
    const double ctas = (double)items * n, tiles = (double)((nt + n - 1) / n);
    const double cost = (5 + tiles * (ctas > 148 ? 4.0 / 3 : 1.0) + 0.25 * n) * (ctas > 296 ? ctas / 296 : 1.0);
    if (n == 1 || cost < best) best = cost, P->n_split = n;
  }
  P->items = items * P->n_split;
}

template <int D>
static cudaError_t launch_cache(const CUtensorMap& mK, const CUtensorMap& mV, const CUtensorMap& mKt,
                                const CUtensorMap& mVt, const CacheAttnParams& p, long long items,
                                cudaStream_t stream) {
  auto kern = attn_cache_kernel<D>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), cache_smem<D>(), p.n_split > 8);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)items), dim3(kCacheThreads), cache_smem<D>(), stream, p.n_split, mK, mV,
                       mKt, mVt, p);
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
