// Runs the general ragged kernel's operand loads (ragged_operand.hpp) on the
// host, for every thread of a workgroup, against matrices whose memory ends (and
// then begins) at a page that cannot be read. Prints the case and fails at the
// first access outside a matrix or wrong value.
#include <signal.h>
#include <stdio.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>

#include "../round_dropless_expert_amd/csrc/ragged_operand.hpp"

namespace {

char g_case[256];

void on_fault(int) {
  const char* m = "access outside the matrix: ";
  (void)!write(1, m, strlen(m));
  (void)!write(1, g_case, strlen(g_case));
  (void)!write(1, "\n", 1);
  _exit(2);
}

constexpr size_t kPage = 4096, kRoom = 1 << 21;
char* g_area;  // kRoom readable bytes between two pages that are not

template <typename T>
T value(int64_t i) { return (T)(float)(1 + i % 1021); }

// One tile of a matrix of `rows` (of c down, of the output along) x `width`,
// rows ld apart, from output index `first` on; c has `count` values.
template <typename T, bool kAlong, int kExt, int kStage>
bool run(int outputs, int count, int64_t ld, int first, int extra_keep, bool at_end) {
  typedef moe::OperandLoads<T, kAlong, kExt, kStage> Op;
  const int rows = kAlong ? outputs : count, width = kAlong ? count : outputs;
  const size_t n = (size_t)(rows - 1) * ld + width;
  if (n * sizeof(T) > kRoom) return fprintf(stderr, "room\n"), false;
  T* m = reinterpret_cast<T*>(at_end ? g_area + kRoom - n * sizeof(T) : g_area);
  for (size_t i = 0; i < n; ++i) m[i] = value<T>((int64_t)i);
  snprintf(g_case, sizeof(g_case),
           "%zu-byte elements, c %s, tile %d, stage %d bytes, %d outputs from %d, %d c, ld %lld, "
           "memory %s there",
           sizeof(T), kAlong ? "along" : "down", kExt, kStage, outputs, first, count,
           (long long)ld, at_end ? "ends" : "begins");
  for (int tid = 0; tid < 256; ++tid) {
    Op op;
    op.set(m + (kAlong ? first * ld : first), ld, outputs - first, first, tid);
    const int keep = op.keep > extra_keep ? op.keep : extra_keep;
    const moe::StageSplit s = moe::split_stages(count, Op::kCk, keep);
    if (s.checked < 0 || s.checked > 2) return printf("stages: %s\n", g_case), false;
    for (int i = 0; i < s.whole + s.checked; ++i) {
      typename Op::regs_t reg;
      const int c0 = i * Op::kCk;
      if (i < s.whole)
        op.load(reg, c0);
      else
        op.load_some(reg, c0, count, tid);
      for (int u = 0; u < Op::kPieces; ++u) {
        const int id = tid + 256 * u, per = kExt * (int)sizeof(T) / 16;
        T got[Op::kV];
        memcpy(got, &reg[u], 16);
        for (int v = 0; v < Op::kV; ++v) {
          const int o = kAlong ? id / Op::kChunks : id % per * Op::kV + v;
          const int c = c0 + (kAlong ? id % Op::kChunks * Op::kV + v : id / per);
          if (first + o >= outputs) continue;  // never stored
          const int64_t at = kAlong ? (first + o) * ld + c : c * ld + first + o;
          const T want = c < count ? m[at] : (T)0.0f;
          if (got[v] != want) return printf("value: %s\n", g_case), false;
        }
      }
    }
  }
  return true;
}

template <typename T, bool kAlong, int kExt, int kStage>
bool tile() {
  constexpr int kCk = kStage / (int)sizeof(T);
  int outputs[32], n_out = 0, counts[64], n_cnt = 0;
  for (int w = 1; w <= 9; ++w) outputs[n_out++] = w;
  for (int w : {kExt - 1, kExt, kExt + 1, kExt + 2, kExt + 7, kExt + 8, 2 * kExt - 3})
    outputs[n_out++] = w;
  for (int c = 1; c <= 9; ++c) counts[n_cnt++] = c;
  for (int c = kCk - 1; c <= kCk + 9; ++c) counts[n_cnt++] = c;
  for (int c : {2 * kCk - 1, 2 * kCk, 2 * kCk + 1, 2 * kCk + 6, 3 * kCk + 3}) counts[n_cnt++] = c;
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < n_cnt; ++j)
      for (int pad : {0, 1, 3, 7, 11})
        for (int first = 0; first < outputs[i]; first += kExt)
          for (int keep : {0, 7})
            for (bool at_end : {true, false}) {
              const int64_t ld = (kAlong ? counts[j] : outputs[i]) + pad;
              if (!run<T, kAlong, kExt, kStage>(outputs[i], counts[j], ld, first, keep, at_end))
                return false;
            }
  return true;
}

template <typename T, bool kAlong>
bool tiles() {
  return tile<T, kAlong, 128, 128>() && tile<T, kAlong, 64, 128>() && tile<T, kAlong, 32, 512>();
}

}  // namespace

int main() {
  char* p = static_cast<char*>(mmap(nullptr, kRoom + 2 * kPage, PROT_READ | PROT_WRITE,
                                    MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
  if (p == MAP_FAILED) return 3;
  mprotect(p, kPage, PROT_NONE);
  mprotect(p + kPage + kRoom, kPage, PROT_NONE);
  g_area = p + kPage;
  signal(SIGSEGV, on_fault);
  signal(SIGBUS, on_fault);
  if (!tiles<_Float16, false>() || !tiles<float, false>() || !tiles<_Float16, true>() ||
      !tiles<float, true>())
    return 1;
  printf("ok\n");
  return 0;
}
