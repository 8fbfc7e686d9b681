// bwd_window_pipeline.cpp -- test infrastructure, host only.  Runs the main kernel
// of the windowed backward (csrc/attn_bwd_window.cu, unchanged) as one CTA of the
// model in sm100.cuh beside this file, under random timings, and checks what every
// product, tensor-memory access and copy finds against the list of (key tile, query
// tile) pairs that the CTA's stretches stand for:
//
//  - a product runs on the tiles of its pair, landed, with P or dS of all warps of
//    that pair and no other, and starts a sum exactly at a walk's first pair;
//  - S, dP and dQ are read once by every warp that needs them before they are
//    overwritten, dK and dV when the products of all the walk's pairs, and none of
//    the next walk's, are in them;
//  - no stage of shared memory is written while something still reads it;
//  - all pairs are done, and no wait is left that nothing completes;
//  - when a copy or a commit is lost, or a wait runs out too early, the CTA still ends,
//    with the abort flag raised.
//
// usage: bwd_window_pipeline d B T G k n_shared sg window sinks trials seed mode
// mode: what is late: copies, commits, products, reads (of the staging
// buffers) or nothing; lost_copy, lost_commit: one of them, another in each trial, never
// comes; timeout: a wait runs out at some step of each trial.
// Prints the first fault and its trial; exit code 1 then.
#include "sm100.cuh"

namespace gqe {
namespace {
alignas(1024) uint8_t smem_raw[1 << 18];
}
}  // namespace gqe

#include "attn_bwd_window.cu"

namespace gqe {
// the padded row space, as attn_bwd.cu lays it out
void attn_bwd_layout(int B, int T, int G, int k, int n_shared, int d, AttnBwdLayout* L) {
  L->rows_pad = (T * k + 127) / 128 * 128;
  L->rows_pad_sh = (T + 127) / 128 * 128;
  L->n_rows_pad = (long long)B * G * L->rows_pad + (n_shared ? (long long)B * L->rows_pad_sh : 0);
  L->off_lse2 = L->off_delta = L->off_dq = 0;
  L->bytes = (size_t)L->n_rows_pad * (d * 4 + 8);
}
}  // namespace gqe

namespace {

using namespace gqe;

struct Pair {
  int s, jt, shared, qi, item;
  bool first, last;
};
std::vector<Pair> pairs;            // of the CTA, in order
std::vector<int> item_end;          // pairs through the end of item i
CUtensorMap maps[7];                // Q, Qs, dO, dOs, K, V, dQ
AttnBwdParams p;
AttnBwdSchedule sched;

struct Box {
  int map = -1, row = -1, seq = -1, col = -1;
  bool landed = false;
};
std::map<uint32_t, Box> boxes;      // by shared-memory address
int s_done, dp_done, dv_steps, dk_steps, dq_steps, s_steps, dp_steps;
int s_reads[16], dp_reads[16], p_writes[16], dst_writes[16], ds_writes[16], dq_reads[16], dk_reads[16], dv_reads[16];
int bulk_landed;

void need(bool ok, const std::string& what) {
  if (!ok) fake::fail(what);
}
bool all(const int* a, int lo, int hi, int v) {
  for (int w = lo; w < hi; ++w)
    if (a[w] != v) return false;
  return true;
}
bool all_from(const int* a, int lo, int hi, int v) {
  for (int w = lo; w < hi; ++w)
    if (a[w] < v) return false;
  return true;
}

template <int D>
struct Model {
  using C = BwdWinCfg<D>;
  static constexpr int kSteps = D / 16;          // k-steps of S and dP; the others have 8

  static void box_is(uint32_t addr, int map, int row, int seq, int col, const char* what) {
    const Box& b = boxes[addr & ~(uint32_t)(kBoxW - 1)];
    need(b.landed && b.map == map && b.row == row && b.seq == seq && b.col == col,
         std::string(what) + ": the operand's tile is not there");
  }
  static int batch(const Pair& x) { return x.s / p.G; }
  static void q_box(const Pair& x, uint32_t addr, int col, bool dO, const char* what) {
    box_is(addr, (dO ? 2 : 0) + x.shared, x.qi * 128, x.shared ? batch(x) : x.s, col, what);
  }
  static const Pair& pair(int n) {
    static const Pair none{};
    if (n >= (int)pairs.size()) {
      fake::fail("a product past the last pair");
      return none;
    }
    return pairs[n];
  }

  static void product(uint32_t d, uint32_t a, bool a_tmem, uint32_t b, bool accumulate) {
    if (d == C::kS) {
      const int n = s_steps / kSteps, ks = s_steps % kSteps;
      const Pair& x = pair(n);
      if (ks == 0) {
        need(all(s_reads, 4, 12, n), "S overwritten before every warp has read it");
        if (C::kWide) need(dv_steps == 8 * n, "S overwrites P that dV has not read");
      }
      need(accumulate == (ks > 0), "S accumulates over another S");
      box_is(a, 4, x.jt * 128, x.s, (ks >> 2) * 64, "S (K)");
      q_box(x, b, (ks >> 2) * 64, false, "S (Q)");
      if (++s_steps % kSteps == 0) ++s_done;
    } else if (d == C::kDP && !(C::kWide && b < (uint32_t)C::OffDO)) {
      const int n = dp_steps / kSteps, ks = dp_steps % kSteps;
      const Pair& x = pair(n);
      if (ks == 0) {
        need(all(dp_reads, 4, 12, 2 * n), "dP overwritten before every warp has read it");
        if (C::kWide) need(all(dq_reads, 12, 16, n), "dP overwrites dQ that was not drained");
        else need(dk_steps == 8 * n, "dP overwrites dS that dK has not read");
      }
      need(accumulate == (ks > 0), "dP accumulates over another dP");
      box_is(a, 5, x.jt * 128, x.s, (ks >> 2) * 64, "dP (V)");
      q_box(x, b, (ks >> 2) * 64, true, "dP (dO)");
      if (++dp_steps % kSteps == 0) ++dp_done;
    } else if (d == C::kDV) {
      const int n = dv_steps / 8, ks = dv_steps % 8;
      const Pair& x = pair(n);
      need(a_tmem && a == C::pt_col(ks < 4 ? 0 : 4) + (ks & 3) * 8, "dV: P's columns");
      need(all(p_writes, 4, 12, n + 1), "dV without every warp's P of its pair");
      if (x.first && ks == 0) need(all(dv_reads, 12, 16, x.item * D / 32), "dV overwritten before it was read");
      need(accumulate == (!x.first || ks > 0), "dV starts at a wrong pair");
      for (int c = 0; c < C::NB; ++c) q_box(x, b + c * kBoxW, c * 64, true, "dV (dO)");
      ++dv_steps;
    } else if (d == C::kDK) {
      const int n = dk_steps / 8, ks = dk_steps % 8;
      const Pair& x = pair(n);
      need(all(ds_writes, 4, 12, 8 * (n + 1)) && (C::kWide || all(dst_writes, 4, 12, 2 * (n + 1))),
           "dK without every warp's dS of its pair");
      need(a_tmem == !C::kWide, "dK: where its dS is");
      if (x.first && ks == 0) need(all(dk_reads, 12, 16, x.item * D / 32), "dK overwritten before it was read");
      need(accumulate == (!x.first || ks > 0), "dK starts at a wrong pair");
      for (int c = 0; c < C::NB; ++c) q_box(x, b + c * kBoxW, c * 64, false, "dK (Q)");
      ++dk_steps;
    } else if (d == C::kDQ) {
      const int n = dq_steps / 8, ks = dq_steps % 8;
      const Pair& x = pair(n);
      if (ks == 0) {
        need(all(dq_reads, 12, 16, n), "dQ overwritten before it was drained");
        if (C::kWide) need(all(dp_reads, 4, 12, 2 * (n + 1)), "dQ overwrites dP that was not read");
      }
      need(all(ds_writes, 4, 12, 8 * (n + 1)), "dQ without every warp's dS of its pair");
      need(accumulate == (ks > 0), "dQ accumulates over another dQ");
      for (int c = 0; c < C::NB; ++c) box_is(b + c * kBoxW, 4, x.jt * 128, x.s, c * 64, "dQ (K)");
      ++dq_steps;
    } else {
      fake::fail("a product into unknown columns");
    }
  }

  static void tmem_load(uint32_t addr, int cols) {
    const int w = fake::current;
    if (w >= 4 && w < 12 && addr < C::kDP && cols == 64) {
      const int n = s_reads[w]++;
      need(s_done == n + 1 && s_steps % kSteps == 0, "S read before it is done, or after it was overwritten");
    } else if (w >= 4 && w < 12 && addr >= C::kDP && addr < C::kDV && cols == 32) {
      const int n = dp_reads[w]++ / 2;
      need(dp_done == n + 1 && dp_steps % kSteps == 0, "dP read before it is done, or after it was overwritten");
    } else if (w >= 12 && addr == C::kDQ && cols == D) {
      const int n = dq_reads[w]++;
      need(dq_steps == 8 * (n + 1), "dQ read before it is done, or after it was overwritten");
    } else if (w >= 12 && addr >= C::kDV && addr < C::kDK && cols == 32) {
      const int i = dv_reads[w]++ / (D / 32);
      need(i < (int)item_end.size() && dv_steps == 8 * item_end[i], "dV read before its walk's last product, or after");
    } else if (w >= 12 && addr >= C::kDK && addr < C::kDK + D && cols == 32) {
      const int i = dk_reads[w]++ / (D / 32);
      need(i < (int)item_end.size() && dk_steps == 8 * item_end[i], "dK read before its walk's last product, or after");
    } else {
      fake::fail("a tensor-memory load of unknown columns");
    }
  }

  static void tmem_store(uint32_t addr, int cols) {
    const int w = fake::current, wg = (w - 4) >> 2;
    if (cols == 32 && addr == C::pt_wcol(wg)) {
      const int n = p_writes[w]++;
      need(dv_steps == 8 * n, "P overwritten before dV has read it");
      // d = 128: P of both warpgroups lies over S of the first
      need(s_reads[w] == n + 1 && (!C::kWide || s_reads[4 + (w & 3)] == n + 1), "P written before S of its pair was read");
    } else if (cols == 16 && addr >= C::dst_wcol(wg) && addr < C::dst_wcol(wg) + 32) {
      const int n = dst_writes[w]++ / 2;
      need(dk_steps == 8 * n, "dS overwritten before dK has read it");
      need(dp_reads[w] == 2 * n + (addr == C::dst_wcol(wg) ? 1 : 2), "dS over dP that was not read");
    } else {
      fake::fail("a tensor-memory store to unknown columns");
    }
  }

  static void store(uint32_t addr) {
    const int w = fake::current;
    if (addr >= C::OffDS && addr < (uint32_t)C::OffEpi) {
      const int n = ds_writes[w]++ / 8;
      need(dq_steps == 8 * n && (!C::kWide || dk_steps == 8 * n), "dS overwritten before its products have read it");
    } else if (addr >= C::OffEpi && addr < (uint32_t)C::OffLse) {
      need(fake::fibers[w].reads == 0, "a staging buffer overwritten while it is stored");
    } else {
      fake::fail("a store to unknown shared memory");
    }
  }

  static void copy(uint32_t dst, const void* map, int c0, int c1, int c2, bool landed) {
    if (!landed) {
      boxes[dst].landed = false;      // whoever still has to read the box finds it gone
    } else {
      boxes[dst] = Box{(int)static_cast<const CUtensorMap*>(map)->opaque[0], c1, c2, c0, true};
    }
  }

  // -LSE2 and -Delta of pair n into stage n & 1: the warps have done pair n - 2
  static void bulk(uint32_t, bool landed) {
    if (!landed) {
      const int n = bulk_landed++ / 2;
      if (n >= 2) need(all_from(ds_writes, 4, 12, 8 * (n - 1)), "-LSE2 or -Delta overwritten while a warp reads them");
    }
  }

  // The pairs of CTA c: walks in the order of sequences and key tiles, cut at the
  // stretches' ends; a query tile is in a key tile's walk when one of its tokens sees
  // one of its keys.
  static void list(int cta) {
    pairs.clear();
    item_end.clear();
    const int n_jt = (p.T + 127) / 128;
    std::vector<Pair> every;
    for (int s = 0; s < p.B * p.G; ++s)
      for (int jt = 0; jt < n_jt; ++jt) {
        const int last_key = jt * 128 + 127;
        const bool sink = jt * 128 < p.sinks;
        for (int sh = 0; sh <= (p.n_shared && s % p.G == p.sg ? 1 : 0); ++sh) {
          const int kk = sh ? 1 : p.k;
          for (int qi = jt * kk; qi * 128 < p.T * kk; ++qi)
            if (sink || qi * 128 / kk < last_key + p.window) every.push_back(Pair{s, jt, sh, qi, 0, false, false});
        }
      }
    long long total = (long long)every.size();
    const int n = sched.n_ctas * sched.n_rounds;
    int item = -1;
    for (int id = cta; id < n; id += sched.n_ctas) {
      const long long lo = total * id / n, hi = total * (id + 1) / n;
      for (long long i = lo; i < hi; ++i) {
        Pair x = every[i];
        x.first = i == lo || every[i - 1].s != x.s || every[i - 1].jt != x.jt;
        x.last = i + 1 == hi || every[i + 1].s != x.s || every[i + 1].jt != x.jt;
        if (x.first) ++item;
        x.item = item;
        pairs.push_back(x);
        if (x.last) item_end.push_back((int)pairs.size());
      }
    }
  }

  static bool trial(int cta, bool losing) {
    list(cta);
    boxes.clear();
    s_done = dp_done = dv_steps = dk_steps = dq_steps = s_steps = dp_steps = bulk_landed = 0;
    for (int* a : {s_reads, dp_reads, p_writes, dst_writes, ds_writes, dq_reads, dk_reads, dv_reads})
      memset(a, 0, 16 * sizeof(int));
    fake::base = smem_raw;
    blockIdx.x = cta;
    bool ok = fake::run_cta(16, [] {
      attn_bwd_window_kernel<D>(maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], maps[6], p, sched);
    });
    const int n = (int)pairs.size();
    fake::current = -1;
    if (ok && losing) {
      const int flag = reinterpret_cast<BwdWinBarriers*>(smem_raw + C::OffBar)->abort;
      if (fake::aborted != (flag != 0)) {
        fake::error = "a wait ran out and the abort flag is down";
        return false;
      }
      if (fake::aborted) return true;       // else nothing waited for what was lost: all must be done
    }
    if (ok && fake::aborted) {
      fake::error = "a wait ran out";
      return false;
    }
    if (ok && !(s_done == n && dp_done == n && dv_steps == 8 * n && dk_steps == 8 * n && dq_steps == 8 * n &&
                all(dq_reads, 12, 16, n) && all(dk_reads, 12, 16, (int)item_end.size() * D / 32) &&
                all(dv_reads, 12, 16, (int)item_end.size() * D / 32))) {
      fake::fail("some pairs were left out");
      ok = false;
    }
    return ok;
  }
};

bool wide;

}  // namespace

void fake::on_product(uint32_t d, uint32_t a, bool a_tmem, uint32_t b, bool acc) {
  wide ? Model<128>::product(d, a, a_tmem, b, acc) : Model<64>::product(d, a, a_tmem, b, acc);
}
void fake::on_tmem_load(uint32_t a, int n) { wide ? Model<128>::tmem_load(a, n) : Model<64>::tmem_load(a, n); }
void fake::on_tmem_store(uint32_t a, int n) { wide ? Model<128>::tmem_store(a, n) : Model<64>::tmem_store(a, n); }
void fake::on_store(uint32_t a) { wide ? Model<128>::store(a) : Model<64>::store(a); }
void fake::on_copy(uint32_t dst, const void* map, int c0, int c1, int c2, bool landed) {
  wide ? Model<128>::copy(dst, map, c0, c1, c2, landed) : Model<64>::copy(dst, map, c0, c1, c2, landed);
}
void fake::on_bulk(uint32_t dst, const void*, uint32_t, bool landed) {
  wide ? Model<128>::bulk(dst, landed) : Model<64>::bulk(dst, landed);
}

int main(int argc, char** argv) {
  if (argc != 13) return 2;
  int v[11];
  for (int i = 0; i < 11; ++i) v[i] = atoi(argv[i + 1]);
  const int d = v[0], trials = v[9], seed = v[10];
  const std::string mode = argv[12];
  p.B = v[1], p.T = v[2], p.G = v[3], p.k = v[4], p.n_shared = v[5], p.sg = v[6], p.window = v[7], p.sinks = v[8];
  p.d = d;
  wide = d == 128;
  AttnBwdLayout L;
  attn_bwd_layout(p.B, p.T, p.G, p.k, p.n_shared, d, &L);
  p.rows_pad = L.rows_pad;
  p.rows_pad_sh = L.rows_pad_sh;
  p.n_rows_pad = L.n_rows_pad;
  size_t off, bytes;
  attn_bwd_window_plan(p.B, p.T, p.G, p.k, p.n_shared, p.sg, d, p.window, p.sinks, &sched, &off, &bytes);
  std::vector<float> part((bytes - off) / 4);
  std::vector<gqe_bf16_t> dK((size_t)p.B * p.G * p.T * d), dV(dK.size());
  for (int i = 0; i < 7; ++i) maps[i].opaque[0] = i;       // the kernel gets copies
  p.part = part.data();
  p.dK = dK.data();
  p.dV = dV.data();
  const double slow = 0.002;
  for (int t = 0; t < trials; ++t) {
    fake::rng.seed(seed + t);
    for (double& w : fake::weight) w = 1.0;
    fake::weight[fake::kProduct] = 4.0;
    if (mode == "copies") fake::weight[fake::kCopy] = slow;
    if (mode == "commits") fake::weight[fake::kCommit] = slow;
    if (mode == "products") fake::weight[fake::kProduct] = 0.02;
    if (mode == "reads") fake::weight[fake::kRead] = slow;
    const int cta = (int)(fake::rng() % (unsigned)sched.n_ctas);
    const bool losing = mode == "lost_copy" || mode == "lost_commit" || mode == "timeout";
    fake::lose_kind = mode == "lost_copy" ? fake::kCopy : fake::kCommit;
    fake::lose = mode != "timeout" && losing ? (int)(fake::rng() % 60u) : -1;
    fake::timeout_at = mode == "timeout" ? (long)(fake::rng() % 6000u) : -1;
    const bool ok = wide ? Model<128>::trial(cta, losing) : Model<64>::trial(cta, losing);
    if (!ok) {
      printf("trial %d, CTA %d of %d, %d pairs in %d walks: %s\n", t, cta, sched.n_ctas, (int)pairs.size(),
             (int)item_end.size(), fake::error.c_str());
      return 1;
    }
  }
  printf("%d trials, %d CTAs, %d rounds\n", trials, sched.n_ctas, sched.n_rounds);
  return 0;
}
