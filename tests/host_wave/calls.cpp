// The attention layer's launches on host arrays (hip/hip_runtime.h beside this
// file), for tests that call them through ctypes.  The sources named here are
// the library's own, with `kernel<<<grid, block, 0, stream>>>(args)` written
// host_launch(kernel, grid, block, args).
#include <setjmp.h>
#include <signal.h>
#include <sys/mman.h>

#include <hip/hip_runtime.h>

#include "nvfp4_attn.hip"
#include "nvfp4_attn_few.hip"
#include "nvfp4_attn_many.hip"
#include "nvfp4_kv_cache.hip"
#include "nvfp4_rope.hip"

threadIdx_t threadIdx;
blockIdx_t blockIdx;
blockDim_t blockDim;
gridDim_t gridDim;

namespace host {

Lane lanes[kMost];
int lane_now;
uint64_t slot[3][kMost], given[3][kMost / 64];
int turn[kMost];

static void* main_sp;
static char* stacks;
static void (*body_now)(void*);
static void* args_now;

// Saves the callee's registers on the stack, leaves the stack pointer in *from and goes on where `to` was left.
extern "C" void host_switch(void** from, void* to);
asm(R"(
.text
.globl host_switch
host_switch:
  pushq %rbp
  pushq %rbx
  pushq %r12
  pushq %r13
  pushq %r14
  pushq %r15
  movq %rsp, (%rdi)
  movq %rsi, %rsp
  popq %r15
  popq %r14
  popq %r13
  popq %r12
  popq %rbx
  popq %rbp
  ret
)");

static void leave(State s) {
  Lane& me = lanes[lane_now];
  me.state = s;
  host_switch(&me.sp, main_sp);
}
void wait(State s) { leave(s); }

static void enter() {
  body_now(args_now);
  leave(kDone);
  abort();
}

static void run(int i) {
  lane_now = i;
  threadIdx = {(unsigned)i, 0, 0};
  lanes[i].state = kRuns;
  host_switch(&main_sp, lanes[i].sp);
}

static void run_block(int n) {
  for (int i = 0; i < n; ++i) {
    void** sp = reinterpret_cast<void**>(stacks + (size_t)(i + 1) * kStack);
    *--sp = nullptr;  // enter() begins as if called: 16-byte aligned but for the return address
    *--sp = reinterpret_cast<void*>(&enter);
    sp -= 6;
    lanes[i] = {sp, kAtWave};
    turn[i] = 0;
  }
  memset(given, 0, sizeof given);
  for (bool more = true; more;) {
    more = false;
    for (int w = 0; w < n; w += 64) {  // each wave up to the barrier or its end
      while (true) {
        int at = 0;
        for (int i = w; i < min(w + 64, n); ++i) {
          if (lanes[i].state == kAtWave) run(i);
          at += lanes[i].state == kAtWave;
        }
        if (at == 0) break;
      }
      int waits = 0, done = 0;
      for (int i = w; i < min(w + 64, n); ++i) {
        waits += lanes[i].state == kAtBarrier;
        done += lanes[i].state == kDone;
      }
      if (waits && done) fprintf(stderr, "host_wave: part of a wave at a barrier\n"), abort();
      more = more || waits;
    }
    for (int i = 0; i < n; ++i)
      if (lanes[i].state == kAtBarrier) lanes[i].state = kAtWave;
  }
}

void launch(dim3 grid, dim3 block, void (*body)(void*), void* args) {
  if (!stacks) stacks = static_cast<char*>(mmap(nullptr, (size_t)kMost * kStack, PROT_READ | PROT_WRITE,
                                                MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  const unsigned n = block.x;
  if (n > kMost || block.y * block.z != 1) abort();
  blockDim = {block.x, block.y, block.z};
  gridDim = {grid.x, grid.y, grid.z};
  body_now = body;
  args_now = args;
  for (unsigned z = 0; z < grid.z; ++z)
    for (unsigned y = 0; y < grid.y; ++y)
      for (unsigned x = 0; x < grid.x; ++x) {
        blockIdx = {x, y, z};
        run_block((int)n);
      }
}

static sigjmp_buf out;
static void* volatile fault_at;
static void on_fault(int, siginfo_t* info, void*) {
  fault_at = info->si_addr;
  siglongjmp(out, 1);
}
// 0, or the address of an access that has no memory.
template <class F>
uint64_t guarded(F f) {
  static char alt[64 << 10];
  stack_t st = {}, old_st;
  st.ss_sp = alt;
  st.ss_size = sizeof alt;
  struct sigaction act = {}, old[2];
  act.sa_sigaction = on_fault;
  act.sa_flags = SA_SIGINFO | SA_ONSTACK;
  sigaltstack(&st, &old_st);
  sigaction(SIGSEGV, &act, &old[0]);
  sigaction(SIGBUS, &act, &old[1]);
  fault_at = nullptr;
  if (sigsetjmp(out, 1) == 0) f();
  sigaction(SIGSEGV, &old[0], nullptr);
  sigaction(SIGBUS, &old[1], nullptr);
  sigaltstack(&old_st, nullptr);
  return reinterpret_cast<uint64_t>(fault_at);
}

}  // namespace host

// What the ranges of a call would do, without doing it: a workgroup of one wave per range.
namespace nvfp4 {
struct Piece {
  int64_t range, seq, tile, minor, k0, k1, slot, steps;  // steps: of the unit's rows, from its first key
};
static void pieces_kernel(Attn a, int rows, Piece* out, int most, int* n) {
  run_range(a, blockIdx.x, [&](const Unit& u, int k0, int k1, int slot) {
    if (threadIdx.x == 0) {
      if (*n < most) out[*n] = {(int64_t)blockIdx.x, u.seq, u.tile, u.minor, k0, k1, slot, reach_of(a, u, rows, 0, rows).steps};
      ++*n;
    }
  });
}
}  // namespace nvfp4

extern "C" {

// `bytes` between unmapped pages, at the beginning of the mapped ones or (at_end) at their end.
void* host_alloc(uint64_t bytes, int at_end) {
  const uint64_t page = 4096, room = (bytes + page - 1) / page * page;
  char* p = static_cast<char*>(mmap(nullptr, room + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  if (p == MAP_FAILED) return nullptr;
  if (room) mprotect(p + page, room, PROT_READ | PROT_WRITE);
  return p + page + (at_end ? room - bytes : 0);
}

void host_free(void* p, uint64_t bytes) {
  const uint64_t page = 4096, at = reinterpret_cast<uint64_t>(p) / page * page;
  munmap(reinterpret_cast<void*>(at - page), (bytes + page - 1) / page * page + 2 * page);
}

uint64_t host_attn_workspace(int64_t T, int n_seqs, int hq, int hk, int d) {
  return nvfp4::attn_cached_workspace_bytes(T, n_seqs, hq, hk, d);
}

// rows, ranges, whether each wave has a range, of a call's layout.
void host_attn_plan(int64_t T, int n_seqs, int hk, int group, int d, int* out) {
  const nvfp4::Plan p = nvfp4::plan_of(T, n_seqs, hk, group, d);
  out[0] = p.rows;
  out[1] = p.ranges;
  out[2] = p.solo;
}

uint64_t host_attn(uint8_t* k, uint8_t* v, uint8_t* ks, uint8_t* vs, const float* k_gs, const float* v_gs, int fp4,
                   int n_pages, int page_shift, int hk, int d, const int32_t* table, int64_t ld_table, int max_pages,
                   const int32_t* lens, const int32_t* cu, int n_seqs, int64_t T, const void* q, int64_t ldq, int hq,
                   float scale, const uint64_t* tree, void* o, int64_t ldo, void* workspace) {
  const nvfp4::KvCache c{k, v, ks, vs, k_gs, v_gs, fp4 != 0, n_pages, page_shift, hk, d};
  const nvfp4::KvRows r{table, ld_table, max_pages, lens, cu, n_seqs, T};
  return host::guarded([&] { nvfp4::launch_attn_cached(c, r, q, ldq, hq, scale, tree, o, ldo, workspace, nullptr); });
}

uint64_t host_kv(int write, uint8_t* k, uint8_t* v, uint8_t* ks, uint8_t* vs, const float* k_gs, const float* v_gs, int fp4,
                 int n_pages, int page_shift, int hk, int d, const int32_t* table, int64_t ld_table, int max_pages,
                 const int32_t* lens, const int32_t* cu, int n_seqs, int64_t T, void* rk, void* rv, int64_t ld, int bf16) {
  const nvfp4::KvCache c{k, v, ks, vs, k_gs, v_gs, fp4 != 0, n_pages, page_shift, hk, d};
  const nvfp4::KvRows r{table, ld_table, max_pages, lens, cu, n_seqs, T};
  return host::guarded([&] {
    if (write)
      nvfp4::launch_kv_cache_write(c, r, rk, ld, rv, ld, bf16 != 0, nullptr);
    else
      nvfp4::launch_kv_cache_read(c, r, rk, ld, rv, ld, bf16 != 0, nullptr);
  });
}

uint64_t host_rope(const void* x, int bf16, int64_t ldx, int64_t q_col, int64_t k_col, int64_t T, int hq, int hk, int d,
                   int rot, const float* q_w, const float* k_w, float eps, const float* table, int n_pos, const int32_t* pos,
                   int n_axes, const uint32_t* axis, int adjacent, uint16_t* q, uint16_t* k) {
  nvfp4::QkNormRope a{x,   bf16 != 0, ldx,   q_col, k_col,  T,  hq,           hk, d,          rot, q_w, k_w,
                      eps, table,     n_pos, pos,   n_axes, {}, adjacent != 0, q,  (int64_t)hq * d, k, (int64_t)hk * d};
  memcpy(a.axis, axis, sizeof a.axis);
  return host::guarded([&] { nvfp4::launch_qk_norm_rope(a, nullptr); });
}

// Pieces of work [most][8] of a call (their number is returned): rows and lengths as for host_attn, no cache.
int host_attn_pieces(int page_shift, int hk, int d, int max_pages, const int32_t* lens, const int32_t* cu, int n_seqs,
                     int64_t T, int hq, int tree, int64_t* out, int most) {
  const nvfp4::KvCache c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, false, 1, page_shift, hk, d};
  const nvfp4::KvRows r{nullptr, max_pages, max_pages, lens, cu, n_seqs, T};
  const nvfp4::Plan p = nvfp4::plan_of(T, n_seqs, hk, hq / hk, d);
  uint64_t mask = 0;  // whether there is one is all that places depend on
  void* ws = calloc(1, nvfp4::attn_cached_workspace_bytes(T, n_seqs, hq, hk, d));
  const nvfp4::Attn a = nvfp4::attn_of(p, c, r, nullptr, 0, hq / hk, 1.0f, tree ? &mask : nullptr, nullptr, 0, ws);
  int n = 0;
  host_launch(nvfp4::pieces_kernel, dim3(p.ranges), dim3(64), a, p.rows, reinterpret_cast<nvfp4::Piece*>(out), most, &n);
  free(ws);
  return n;
}

}  // extern "C"
