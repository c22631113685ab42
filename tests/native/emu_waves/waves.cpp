// The workgroups of a launch on the CPU, one after another: a coroutine for
// each lane, run in the order of the lanes within a wave and of the waves (or
// against it, so that a missing barrier shows in the results), from one
// operation of the wave or barrier to the next.  Compiled without sanitizers.

#include <hip/hip_runtime.h>
#include <sanitizer/common_interface_defs.h>
#include <sys/mman.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>
#include <vector>

zr_emu_dim zr_emu_block, zr_emu_thread, zr_emu_grid, zr_emu_size;
bool zr_emu_waves_backwards = false;
long long zr_emu_workgroups = 0;

namespace {

constexpr unsigned kMaxLanes = 1024;
constexpr size_t kStack = 512 * 1024;

enum State { kReady, kInWave, kAtBarrier, kDone };
struct Pending {
  void* lds;
  unsigned char data[16];
};
struct Lane {
  void* sp = nullptr;
  char* stack = nullptr;
  State state = kDone;
  zr_emu_op op{};
  unsigned char in[96], out[64];
  std::vector<Pending> later;
};
Lane g_lanes[kMaxLanes];
unsigned g_now;             // the running lane
void* g_scheduler;          // the scheduler's stack pointer
const void* g_bottom;       // and its stack, as the sanitizer wants to know it
size_t g_size;
void (*g_body)(const void*);
const void* g_args;
std::string g_name;

[[noreturn]] void stop(const char* what, unsigned lane) {
  std::fprintf(stderr, "%s: %s (block %u,%u lane %u of %u)\n", g_name.c_str(), what, zr_emu_block.x,
               zr_emu_block.y, lane, zr_emu_size.x);
  std::abort();
}

// Saves the registers a call keeps and the stack pointer, and takes the other's.
extern "C" void zr_emu_switch(void** from, void* to);
asm(R"(
.globl zr_emu_switch
zr_emu_switch:
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

void leave() {   // from the running lane to the scheduler
  Lane& l = g_lanes[g_now];
  void* fake = nullptr;
  __sanitizer_start_switch_fiber(&fake, g_bottom, g_size);
  zr_emu_switch(&l.sp, g_scheduler);
  __sanitizer_finish_switch_fiber(fake, nullptr, nullptr);
}

void lane_main() {
  __sanitizer_finish_switch_fiber(nullptr, &g_bottom, &g_size);
  for (;;) {
    g_body(g_args);
    g_lanes[g_now].state = kDone;
    leave();
  }
}

void enter(unsigned lane) {
  Lane& l = g_lanes[lane];
  if (!l.stack) {
    l.stack = static_cast<char*>(mmap(nullptr, kStack, PROT_READ | PROT_WRITE,
                                      MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
    if (l.stack == MAP_FAILED) stop("no memory for a lane's stack", lane);
    void** top = reinterpret_cast<void**>(l.stack + kStack) - 1;   // as a call leaves it
    *--top = reinterpret_cast<void*>(&lane_main);
    for (int i = 0; i < 6; ++i) *--top = nullptr;
    l.sp = top;
  }
  g_now = lane;
  zr_emu_thread.x = lane;
  void* fake = nullptr;
  __sanitizer_start_switch_fiber(&fake, l.stack, kStack);
  zr_emu_switch(&g_scheduler, l.sp);
  __sanitizer_finish_switch_fiber(fake, nullptr, nullptr);
}

template <typename T>
T in_of(unsigned lane, size_t at = 0) {
  T v;
  std::memcpy(&v, g_lanes[lane].in + at * sizeof(T), sizeof(T));
  return v;
}
template <typename T>
void out_of(unsigned lane, T v) {
  std::memcpy(g_lanes[lane].out, &v, sizeof(T));
}
float widen(uint16_t b) { return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16); }

// What the operation that the lanes of `live` from `base` on have reached gives
// each of them.
void finish(unsigned base, uint64_t live) {
  const unsigned first = base + static_cast<unsigned>(__builtin_ctzll(live));
  const zr_emu_op op = g_lanes[first].op;
  auto there = [&](unsigned lane, unsigned asked) {
    if (lane > 63 || !(live >> lane & 1)) stop("read of a lane that is not there", asked);
    return base + lane;
  };
  uint64_t ballot = 0;
  if (op == kBallot)
    for (unsigned i = 0; i < 64; ++i)
      if ((live >> i & 1) && in_of<int>(base + i)) ballot |= 1ull << i;
  if (op == kMfma) {
    if (~live) stop("a matrix product without all lanes", first);
    static float a[32][16], b[16][32];
    for (unsigned i = 0; i < 64; ++i)
      for (unsigned k = 0; k < 8; ++k) {
        a[i % 32][8 * (i / 32) + k] = widen(in_of<uint16_t>(base + i, k));
        b[8 * (i / 32) + k][i % 32] = widen(in_of<uint16_t>(base + i, 8 + k));
      }
    for (unsigned i = 0; i < 64; ++i) {
      float c[16];
      std::memcpy(c, g_lanes[base + i].in + 32, 64);
      for (unsigned v = 0; v < 16; ++v) {
        const unsigned r = 8 * (v / 4) + v % 4 + 4 * (i / 32);
        for (unsigned k = 0; k < 16; ++k) c[v] += a[r][k] * b[k][i % 32];
      }
      std::memcpy(g_lanes[base + i].out, c, 64);
    }
  }
  if (op == kMfmaFlat) {   // 16 x 16, over 32
    if (~live) stop("a matrix product without all lanes", first);
    static float a[16][32], b[32][16];
    for (unsigned i = 0; i < 64; ++i)
      for (unsigned k = 0; k < 8; ++k) {
        a[i % 16][8 * (i / 16) + k] = widen(in_of<uint16_t>(base + i, k));
        b[8 * (i / 16) + k][i % 16] = widen(in_of<uint16_t>(base + i, 8 + k));
      }
    for (unsigned i = 0; i < 64; ++i) {
      float c[4];
      std::memcpy(c, g_lanes[base + i].in + 32, 16);
      for (unsigned v = 0; v < 4; ++v)
        for (unsigned k = 0; k < 32; ++k) c[v] += a[4 * (i / 16) + v][k] * b[k][i % 16];
      std::memcpy(g_lanes[base + i].out, c, 16);
    }
  }
  for (unsigned i = 0; i < 64; ++i) {
    if (!(live >> i & 1)) continue;
    const unsigned lane = base + i;
    if (g_lanes[lane].op != op) stop("lanes of a wave at different operations", lane);
    const int x = in_of<int>(lane);
    switch (op) {
      case kFirstLane: out_of(lane, in_of<int>(first)); break;
      case kReadLane: out_of(lane, in_of<int>(there(static_cast<unsigned>(in_of<int>(lane, 1)), lane))); break;
      case kBallot: out_of(lane, ballot); break;
      case kShiftUp: {
        const unsigned d = static_cast<unsigned>(in_of<int>(lane, 1));
        out_of(lane, i >= d ? in_of<int>(there(i - d, lane)) : x);
        break;
      }
      case kQuadPerm: {
        const int control = in_of<int>(lane, 1);
        if (control < 0 || control > 255) stop("not a permutation of four lanes", lane);
        out_of(lane, in_of<int>(there((i & ~3u) + (control >> (2 * (i & 3)) & 3), lane)));
        break;
      }
      case kExchange:
        out_of(lane, in_of<int>(there(i ^ static_cast<unsigned>(in_of<int>(lane, 1)), lane)));
        break;
      case kSwapRows: {
        // rows of sixteen lanes: the odd ones' first for the even ones' second
        int r[2];
        r[0] = i & 16 ? in_of<int>(there(i - 16, lane), 1) : x;
        r[1] = i & 16 ? in_of<int>(lane, 1) : in_of<int>(there(i + 16, lane));
        std::memcpy(g_lanes[lane].out, r, 8);
        break;
      }
      case kTranspose: {
        short r[4];
        for (unsigned j = 0; j < 4; ++j)
          r[j] = in_of<short>(there((i & ~15u) + 4 * j + (i & 15) / 4, lane), i % 4);
        std::memcpy(g_lanes[lane].out, r, 8);
        break;
      }
      default: break;
    }
    g_lanes[lane].state = kReady;
  }
}

// Runs the wave of `lanes` lanes from `base` on until none is ready.
void run_wave(unsigned base, unsigned lanes) {
  for (;;) {
    for (unsigned i = 0; i < lanes; ++i)
      if (g_lanes[base + i].state == kReady) enter(base + i);
    uint64_t live = 0, waiting = 0;
    for (unsigned i = 0; i < lanes; ++i) {
      if (g_lanes[base + i].state != kDone) live |= 1ull << i;
      if (g_lanes[base + i].state == kInWave) waiting |= 1ull << i;
    }
    if (!waiting) return;
    if (waiting != live) stop("some lanes of a wave at a barrier, some not", base);
    finish(base, live);
  }
}

void run_workgroup(unsigned block) {
  const unsigned waves = (block + 63) / 64;
  for (unsigned i = 0; i < block; ++i) {
    g_lanes[i].state = kReady;
    g_lanes[i].later.clear();
  }
  for (;;) {
    for (unsigned k = 0; k < waves; ++k) {
      const unsigned w = zr_emu_waves_backwards ? waves - 1 - k : k;
      run_wave(64 * w, block - 64 * w < 64 ? block - 64 * w : 64);
    }
    bool left = false;
    for (unsigned i = 0; i < block; ++i)
      if (g_lanes[i].state == kAtBarrier) g_lanes[i].state = kReady, left = true;
    if (!left) return;
  }
}

}  // namespace

// Launches per kernel instantiation, named by the sanitizer runtime's
// symbolizer from the kernel's address.
std::map<std::string, long long>& zr_emu_coverage() {
  static std::map<std::string, long long> c;
  return c;
}
static std::string name_of(void* kernel) {
  static std::map<void*, std::string> names;
  auto it = names.find(kernel);
  if (it != names.end()) return it->second;
  char buf[1024] = {0};
  __sanitizer_symbolize_pc(static_cast<char*>(kernel) + 1, "%f", buf, sizeof(buf));
  std::string n(buf);
  const std::string anon = "(anonymous namespace)::";
  const size_t at = n.find(anon);
  if (at != std::string::npos) n = n.substr(at + anon.size());
  size_t end = n.find('(');
  const size_t lt = n.find('<');
  if (lt < end) end = n.rfind('>') + 1;
  n = n.substr(0, end);
  return names.emplace(kernel, n).first->second;
}

void zr_emu_run(dim3 grid, unsigned block, void* kernel, void (*body)(const void*), const void* args) {
  g_name = name_of(kernel);
  ++zr_emu_coverage()[g_name];
  if (!grid.x || !grid.y || !block || block > kMaxLanes) stop("not a launch shape", 0);
  g_body = body;
  g_args = args;
  zr_emu_grid = {grid.x, grid.y, 1};
  zr_emu_size = {block, 1, 1};
  for (unsigned y = 0; y < grid.y; ++y)
    for (unsigned x = 0; x < grid.x; ++x) {
      zr_emu_block = {x, y, 0};
      run_workgroup(block);
      ++zr_emu_workgroups;
    }
}

void zr_emu_wave(zr_emu_op op, const void* in, size_t in_bytes, void* out, size_t out_bytes) {
  Lane& l = g_lanes[g_now];
  l.op = op;
  if (in_bytes) std::memcpy(l.in, in, in_bytes);
  l.state = kInWave;
  leave();
  if (out_bytes) std::memcpy(out, l.out, out_bytes);
}
void zr_emu_barrier() {
  g_lanes[g_now].state = kAtBarrier;
  leave();
}
void zr_emu_lds_later(void* lds, const void* data) {
  Pending p{static_cast<char*>(lds) + 16 * (g_now % 64), {}};
  std::memcpy(p.data, data, 16);
  g_lanes[g_now].later.push_back(p);
}
void zr_emu_wait(unsigned left) {
  std::vector<Pending>& later = g_lanes[g_now].later;
  const size_t there = later.size() > left ? later.size() - left : 0;
  for (size_t k = 0; k < there; ++k) std::memcpy(later[k].lds, later[k].data, 16);
  later.erase(later.begin(), later.begin() + static_cast<std::ptrdiff_t>(there));
}

// e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities.
float zr_emu_e4m3_value(uint8_t code) {
  const int e = code >> 3 & 15, m = code & 7;
  float v = e == 15 && m == 7 ? NAN : e == 0 ? std::ldexp(m, -9) : std::ldexp(8 + m, e - 10);
  return code & 0x80 ? -v : v;
}
uint8_t zr_emu_e4m3(float x) {
  const uint8_t sign = std::signbit(x) ? 0x80 : 0;
  if (std::isnan(x)) return 0x7f;
  const float a = std::fabs(x);
  int e = a > 0 ? std::ilogb(a) : -6;
  if (e < -6) e = -6;
  int q = static_cast<int>(std::nearbyint(std::ldexp(a, 3 - e)));   // 8..16, or a subnormal's 0..8
  if (q == 16) q = 8, ++e;
  if (e > 8 || (e == 8 && q == 15)) return sign | 0x7f;
  return sign | (q < 8 ? q : (e + 7) << 3 | (q & 7));
}

extern "C" {
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "emulated runtime"; }
}
