// sm100.cuh (stand-in) -- test infrastructure, host only.  The device wrappers of
// csrc/sm100.cuh that the attention's backward kernels use, over a small model of one CTA,
// so that a kernel's roles run on a machine without a GPU and the order of their
// waits can be checked under any timing:
//
//  - each warp is a fiber; one lane (lane 0) stands for the warp, so an arrival
//    that every lane makes counts 32.  Any fiber that is not blocked may run next.
//  - mbarriers have PTX's phases: a wait for a parity returns when the phase of
//    that parity is the last completed one, whichever phase the caller means.
//  - when nothing else can happen (or at a step that the harness chooses), a wait runs
//    out: it raises the kernel's abort flag, and the checks on data stop, but the warps
//    must still all come to the end.
//  - copies land, products run and commits arrive as events of their own, at any
//    time after they were issued: a thread's products run in the order of issue, a
//    commit's arrival comes at any time after the thread's earlier products, and the
//    arrivals of two commits in any order.
//
// The harness that includes the kernel gets every product, tensor-memory access,
// copy and store through the hooks below, and checks what each of them finds.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <ucontext.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <functional>
#include <map>
#include <random>
#include <string>
#include <vector>

namespace fake {

// ---------------------------------------------------------------- the CTA
struct Barrier {
  int count = 0, pending = 0;
  long tx = 0;
  unsigned phase = 0;      // completed phases
};

struct Event {
  int kind;                // kCopy, kCommit, kRead
  std::function<void()> run;
};
enum { kCopy, kCommit, kRead, kProduct, kFiber, kKinds };

struct Fiber {
  ucontext_t ctx;
  std::vector<char> stack;
  bool done = false;
  std::function<bool()> blocked_on;          // empty: runnable
  volatile int* abort = nullptr;             // in a bounded wait: the flag it raises when it runs out
  std::deque<std::function<bool()>> queue;   // products (false) and commits (true) issued, in order
  int reads = 0;                             // bulk stores that still read shared memory
};

inline std::vector<Fiber> fibers;
inline std::vector<Event> events;
inline std::map<const void*, Barrier> barriers;
inline ucontext_t main_ctx;
inline int current = -1;
inline std::mt19937 rng;
inline double weight[kKinds];
inline std::string error;
inline std::vector<uint8_t> smem;            // the CTA's shared memory, 1024-byte aligned at `base`
inline uint8_t* base = nullptr;

inline bool aborted = false;                 // some wait has run out
inline int lose = -1;                        // the copy or commit that never comes
inline int lose_kind = kCopy;
inline long timeout_at = -1;                 // step at which a wait runs out although it would have ended
inline bool lost(int kind) { return kind == lose_kind && lose-- == 0; }

inline void fail(const std::string& what) {
  if (error.empty() && !aborted) error = "warp " + std::to_string(current) + ": " + what;
}
inline void yield() { swapcontext(&fibers[current].ctx, &main_ctx); }
inline void block(std::function<bool()> until) {
  fibers[current].blocked_on = std::move(until);
  yield();
}
inline void arrive(const void* b, int n, long tx_add = 0) {
  Barrier& m = barriers[b];
  if (m.count == 0) fail("an arrival on a barrier that was not initialised");
  m.tx += tx_add;
  m.pending -= n;
  if (m.pending < 0) fail("more arrivals in a phase than the barrier counts");
}
inline void settle(const void* b) {
  Barrier& m = barriers[b];
  if (m.pending == 0 && m.tx == 0) {
    ++m.phase;
    m.pending = m.count;
  }
}
inline bool passed(const void* b, uint32_t parity) { return (barriers[b].phase & 1) != (parity & 1); }

// __syncthreads and named barriers: all of n warps have come
struct Meet {
  int come = 0, gen = 0;
  bool any = false, result = false;
};
inline std::map<int, Meet> meets;
inline bool meet(int id, int warps, bool pred) {
  Meet& m = meets[id];
  m.any = m.any || pred;
  const int gen = m.gen;
  if (++m.come == warps) {
    m.come = 0;
    m.result = m.any;
    m.any = false;
    ++m.gen;
  } else {
    block([id, gen] { return meets[id].gen != gen; });
  }
  const bool r = meets[id].result;
  yield();
  return r;
}

// Runs `body` as n warps to the end.  False: stuck, or a check failed.
inline void entry(int lo, int hi) {
  auto* f = reinterpret_cast<std::function<void()>*>(((uintptr_t)(unsigned)hi << 32) | (unsigned)lo);
  (*f)();
  fibers[current].done = true;
  yield();
}
inline void set_thread(int warp);
inline bool run_cta(int n, std::function<void()> body) {
  fibers.clear();
  fibers.resize(n);
  events.clear();
  barriers.clear();
  meets.clear();
  error.clear();
  aborted = false;
  for (Fiber& f : fibers) {
    f.stack.resize(256 * 1024);
    getcontext(&f.ctx);
    f.ctx.uc_stack.ss_sp = f.stack.data();
    f.ctx.uc_stack.ss_size = f.stack.size();
    f.ctx.uc_link = &main_ctx;
    const uintptr_t p = reinterpret_cast<uintptr_t>(&body);
    makecontext(&f.ctx, reinterpret_cast<void (*)()>(entry), 2, (int)(unsigned)p, (int)(unsigned)(p >> 32));
  }
  struct Choice {
    int kind, index;
  };
  std::vector<Choice> can;
  while (error.empty()) {
    can.clear();
    bool all_done = true;
    double total = 0;
    auto offer = [&](int kind, int index) {
      can.push_back({kind, index});
      total += weight[kind];
    };
    for (int i = 0; i < n; ++i) {
      Fiber& f = fibers[i];
      all_done = all_done && f.done;
      if (!f.done && (!f.blocked_on || f.blocked_on())) offer(kFiber, i);
      if (!f.queue.empty()) offer(kProduct, i);
    }
    for (size_t i = 0; i < events.size(); ++i) offer(events[i].kind, (int)i);
    if (can.empty() && all_done) break;
    const bool early = timeout_at >= 0 && timeout_at-- == 0;
    if (can.empty() || early) {
      std::vector<int> waits;
      std::string who;
      for (int i = 0; i < n; ++i)
        if (!fibers[i].done) {
          who += " " + std::to_string(i);
          if (fibers[i].abort) waits.push_back(i);
        }
      if (waits.empty() && can.empty()) {
        error = "stuck: warps" + who + " wait for what nothing brings";
        break;
      }
      if (waits.empty()) {
        timeout_at = 0;      // at the next step, then
      } else {
        aborted = true;
        *fibers[waits[rng() % waits.size()]].abort = 1;
        continue;
      }
    }
    double x = std::uniform_real_distribution<double>(0, total)(rng);
    size_t c = 0;
    while (c + 1 < can.size() && (x -= weight[can[c].kind]) > 0) ++c;
    const Choice ch = can[c];
    if (ch.kind == kFiber) {
      current = ch.index;
      fibers[ch.index].blocked_on = nullptr;
      set_thread(current);
      swapcontext(&main_ctx, &fibers[ch.index].ctx);
    } else if (ch.kind == kProduct) {
      current = ch.index;
      auto op = std::move(fibers[ch.index].queue.front());
      fibers[ch.index].queue.pop_front();
      op();
    } else {
      current = -1;
      auto run = std::move(events[ch.index].run);
      events.erase(events.begin() + ch.index);
      run();
    }
  }
  return error.empty();
}

// ---------------------------------------------------------------- hooks of the harness
void on_copy(uint32_t dst, const void* map, int c0, int c1, int c2, bool landed);   // 128 x 64 box, issued / landed
void on_bulk(uint32_t dst, const void* src, uint32_t bytes, bool landed);
void on_product(uint32_t d, uint32_t a, bool a_tmem, uint32_t b, bool accumulate);  // it runs now
void on_tmem_load(uint32_t addr, int cols);
void on_tmem_store(uint32_t addr, int cols);
void on_store(uint32_t addr);                                                       // 16 bytes of shared memory

}  // namespace fake

// ---------------------------------------------------------------- CUDA's own names
#define __launch_bounds__(...)
inline uint3 threadIdx, blockIdx;
inline dim3 blockDim, gridDim;
inline void fake::set_thread(int warp) { threadIdx.x = warp * 32; }
inline void __syncthreads() { fake::meet(-1, (int)fake::fibers.size(), false); }
inline void __syncwarp(unsigned = ~0u) {}
inline float __shfl_xor_sync(unsigned, float v, int) { return v; }
inline float __uint_as_float(uint32_t v) {
  float f;
  memcpy(&f, &v, 4);
  return f;
}
using std::max;
using std::min;

namespace gqe {

enum DeviceErrorCode : unsigned { kErrTimeoutAttnBwd = 0x202 };

inline uint32_t smem_u32(const void* p) { return (uint32_t)(static_cast<const uint8_t*>(p) - fake::base); }
inline bool elect_one() { return true; }
inline void pdl_wait() {}
inline void pdl_launch_dependents() {}
template <int N>
inline void set_regs_up() {}
template <int N>
inline void set_regs_down() {}

inline void mbar_init(uint64_t* bar, uint32_t count) {
  fake::Barrier& m = fake::barriers[bar];
  m = fake::Barrier{};
  m.count = m.pending = (int)count;
}
inline void fence_mbar_init() {}
inline void mbar_arrive(uint64_t* bar) {
  fake::yield();
  fake::arrive(bar, 32);
  fake::settle(bar);
  fake::yield();
}
inline void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  fake::arrive(bar, 1, bytes);
  fake::settle(bar);
}
inline bool mbar_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const int who = fake::current;
  fake::fibers[who].abort = abort;
  fake::block([=] { return fake::passed(bar, parity) || *abort; });
  fake::fibers[who].abort = nullptr;
  return fake::passed(bar, parity);
}
inline bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned*, unsigned) {
  return mbar_wait_short(bar, parity, abort);
}
inline bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_wait_short(bar, parity, abort);
}
template <int ID, int N>
inline bool bar_or(bool pred) {
  return fake::meet(ID, N / 32, pred);
}
inline void report_abort(volatile int*, unsigned*, unsigned) {}
inline void drain_after_abort(volatile int*) {}
inline void fence_proxy_async_smem() {}
inline void tc_fence_before() {}
inline void tc_fence_after() {}

inline void tma_prefetch_desc(const CUtensorMap*) {}
inline void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  const uint32_t d = smem_u32(dst);
  fake::on_copy(d, map, c0, c1, c2, false);
  if (fake::lost(fake::kCopy)) return;
  fake::events.push_back({fake::kCopy, [=] {
                            fake::on_copy(d, map, c0, c1, c2, true);
                            fake::barriers[bar].tx -= 128 * 128;
                            fake::settle(bar);
                          }});
  fake::yield();
}
inline void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  const uint32_t d = smem_u32(dst);
  fake::on_bulk(d, src, bytes, false);
  fake::events.push_back({fake::kCopy, [=] {
                            fake::on_bulk(d, src, bytes, true);
                            fake::barriers[bar].tx -= bytes;
                            fake::settle(bar);
                          }});
}
inline void tma_reduce_add_2d(const CUtensorMap*, const void*, int, int) {
  const int who = fake::current;
  ++fake::fibers[who].reads;
  fake::events.push_back({fake::kRead, [who] { --fake::fibers[who].reads; }});
}
inline void bulk_commit() {}
template <int N>
inline void bulk_wait_read() {
  const int who = fake::current;
  fake::block([who] { return fake::fibers[who].reads == 0; });
}
template <int N>
inline void bulk_wait() {
  bulk_wait_read<N>();
}
inline void st_shared_v4(void* p, uint32_t, uint32_t, uint32_t, uint32_t) { fake::on_store(smem_u32(p)); }

inline void tmem_alloc(uint32_t* dst, uint32_t) { *dst = 0; }
inline void tmem_dealloc(uint32_t, uint32_t) {}
constexpr uint32_t idesc_bf16_f32(int, int, bool, bool) { return 0; }
inline uint64_t sdesc_sw128(uint32_t saddr, uint32_t, uint32_t) { return saddr; }
inline uint64_t sdesc_at(uint64_t desc, uint32_t bytes) { return desc + bytes; }
inline void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t, uint32_t accumulate) {
  fake::fibers[fake::current].queue.push_back([=] {
    fake::on_product(d, (uint32_t)a, false, (uint32_t)b, accumulate != 0);
    return false;
  });
}
inline void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t, uint32_t accumulate) {
  fake::fibers[fake::current].queue.push_back([=] {
    fake::on_product(d, a, true, (uint32_t)b, accumulate != 0);
    return false;
  });
}
inline void umma_commit(uint64_t* bar) {
  if (fake::lost(fake::kCommit)) return;
  fake::fibers[fake::current].queue.push_back([=] {
    fake::events.push_back({fake::kCommit, [=] {
                              fake::arrive(bar, 1);
                              fake::settle(bar);
                            }});
    return true;
  });
  fake::yield();
}
template <int N>
inline void tmem_ld(uint32_t a, uint32_t* r) {
  fake::yield();
  fake::on_tmem_load(a & 0xFFFFu, N);
  memset(r, 0, N * 4);
  fake::yield();
}
inline void tmem_ld16(uint32_t a, uint32_t* r) { tmem_ld<16>(a, r); }
inline void tmem_ld16_async(uint32_t a, uint32_t* r) { tmem_ld<16>(a, r); }
inline void tmem_wait_ld16(uint32_t*) {}
inline void tmem_st8(uint32_t a, const uint32_t*) { fake::on_tmem_store(a & 0xFFFFu, 8); }
inline void tmem_ld32(uint32_t a, uint32_t* r) { tmem_ld<32>(a, r); }
inline void tmem_ld64(uint32_t a, uint32_t* r) { tmem_ld<64>(a, r); }
inline void tmem_st16(uint32_t a, const uint32_t*) { fake::on_tmem_store(a & 0xFFFFu, 16); }
inline void tmem_st32(uint32_t a, const uint32_t*) { fake::on_tmem_store(a & 0xFFFFu, 32); }
inline void tmem_wait_st() { fake::yield(); }

inline float ex2(float x) { return std::exp2(x); }
inline unsigned long long f2_pack(float a, float) { return (unsigned long long)(a != 0.f); }
inline void f2_unpack(unsigned long long, float& a, float& b) { a = b = 0.f; }
inline unsigned long long f2_fma(unsigned long long a, unsigned long long, unsigned long long) { return a; }
inline unsigned long long f2_add(unsigned long long a, unsigned long long) { return a; }
inline unsigned long long f2_mul(unsigned long long a, unsigned long long) { return a; }
inline uint32_t pack_bf16x2(float, float) { return 0; }
inline float bf16_lo(uint32_t) { return 0.f; }
inline float bf16_hi(uint32_t) { return 0.f; }

}  // namespace gqe
