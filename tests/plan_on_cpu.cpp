// The plan of kv_attend_tree's tile kernel, run on the CPU: SHARES is a file with the kernel's own source of it (tiles, costs, make_plan),
// compiled here with the CTA's threads as fibers and the warp operations as exchanges between them.
//
// Input: G H N CTAs T, then T sequences and T positions.  Every CTA makes its plan and walks through its share as the kernel's
// walking warp does; a line is printed for every unit (tile, kv head) whose blocks are not each held by one CTA, or whose parts are
// not where its Join says.
#include <ucontext.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __noinline__
#define __restrict__
using std::max;
using std::min;

constexpr int KV_BLOCK = 64;

namespace fibers {
constexpr int MOST = 512, STACK = 64 * 1024;
ucontext_t home, at[MOST];
char stack[MOST][STACK];
int now, alive;
struct Meet {   // all of `n` fibers have arrived
  int count = 0;
  unsigned turn = 0;
};
Meet cta, warps[MOST / 32];
uint64_t slots[2][MOST];
void yield() { swapcontext(&at[now], &home); }
unsigned meet(Meet& m, int n) {
  const unsigned turn = m.turn;
  if (++m.count == n) m.count = 0, ++m.turn;
  else
    while (m.turn == turn) yield();
  return turn;
}
// what the warp's lanes give; a lane is never two exchanges ahead of another
template <typename T>
const uint64_t* exchange(T v) {
  Meet& m = warps[now / 32];
  slots[m.turn & 1][now] = (uint64_t)v;
  const unsigned turn = meet(m, 32);
  return slots[turn & 1] + now / 32 * 32;
}
}  // namespace fibers

struct Dim {
  struct X {
    operator int() const { return fibers::now; }
  } x;
} threadIdx;
struct {
  int x;
} blockIdx, gridDim;
void __syncthreads() { fibers::meet(fibers::cta, fibers::MOST); }
uint32_t __ballot_sync(uint32_t, bool p) {
  const uint64_t* v = fibers::exchange(p);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r |= (uint32_t)(v[i] & 1) << i;
  return r;
}
int __reduce_max_sync(uint32_t, int x) {
  const uint64_t* v = fibers::exchange(x);
  int r = INT_MIN;
  for (int i = 0; i < 32; ++i) r = max(r, (int)v[i]);
  return r;
}
uint32_t __reduce_add_sync(uint32_t, uint32_t x) {
  const uint64_t* v = fibers::exchange(x);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r += (uint32_t)v[i];
  return r;
}
template <typename T>
T __shfl_up_sync(uint32_t, T x, int by) {
  const uint64_t* v = fibers::exchange(x);
  const int lane = fibers::now & 31;
  return lane >= by ? (T)v[lane - by] : x;
}
int __clz(uint32_t x) { return x ? __builtin_clz(x) : 32; }
template <typename T>
T __ldg(const T* p) { return *p; }
void atomicMax(int* p, int v) { *p = max(*p, v); }

struct KvTable {
  int N;
};
struct TreeParams {
  int H, G, per, T;
  KvTable tab;
  const int *seq, *pos;
};

#include SHARES

TreeParams a;
PlanMem mem;
void thread() {
  make_plan(a, mem);
  --fibers::alive;
  while (true) fibers::yield();
}

struct Part {
  int cta, b0, b1, slot;
};
struct Join {
  int t0, n, h, parts;
};

int main() {
  int ctas;
  if (scanf("%d %d %d %d %d", &a.G, &a.H, &a.tab.N, &ctas, &a.T) != 5) return 2;
  std::vector<int> seq(a.T), pos(a.T);
  for (int& x : seq) if (scanf("%d", &x) != 1) return 2;
  for (int& x : pos) if (scanf("%d", &x) != 1) return 2;
  a.seq = seq.data(), a.pos = pos.data(), a.per = 2 * (128 / a.G);
  const int per_one = 128 / a.G;
  using Key = std::tuple<int, int, int>;   // first token, tokens, kv head
  std::map<Key, std::vector<Part>> units;
  std::map<Key, int> blocks;
  auto tile = [&](int t0, int* top) {
    int n = 0;
    *top = INT_MIN;
    while (n < a.per && t0 + n < a.T && !other_run(seq[t0], pos[t0], seq[t0 + n], pos[t0 + n])) *top = max(*top, pos[t0 + n++]);
    return n;
  };
  for (int t0 = 0, top; t0 < a.T;) {
    const int n = tile(t0, &top);
    for (int h = 0; h < a.H; ++h) blocks[{t0, n, h}] = top < 0 ? 1 : min(top / KV_BLOCK + 1, a.tab.N);
    t0 += n;
  }
  std::vector<Join> joins(ctas, Join{0, 0, 0, 0});
  gridDim.x = ctas;
  for (int c = 0; c < ctas; ++c) {
    blockIdx.x = c;
    fibers::alive = fibers::MOST;
    for (int i = 0; i < fibers::MOST; ++i) {
      getcontext(&fibers::at[i]);
      fibers::at[i].uc_stack.ss_sp = fibers::stack[i], fibers::at[i].uc_stack.ss_size = fibers::STACK, fibers::at[i].uc_link = nullptr;
      makecontext(&fibers::at[i], thread, 0);
    }
    while (fibers::alive)
      for (fibers::now = 0; fibers::now < fibers::MOST; ++fibers::now) swapcontext(&fibers::home, &fibers::at[fibers::now]);
    const long long lo = mem.lo, hi = mem.hi, share = mem.per;
    if (lo >= hi) continue;
    long long at = mem.found_at;
    for (int t0 = mem.found, top; t0 < a.T && at < hi;) {
      const int n = tile(t0, &top);
      const Unit unit(n, top, a.tab.N, per_one);
      for (int h = 0; h < a.H; ++h, at += unit.cost()) {
        if (at + unit.cost() <= lo) continue;
        if (at >= hi) break;
        const int b0 = unit.first_from(lo - at), b1 = unit.first_from(hi - at);
        if (b0 >= b1) continue;
        int slot = -1;
        if (b0 > 0) slot = 2 * c;
        else if (b1 < unit.blocks) slot = 2 * c + 1, joins[c] = {t0, n, h, (int)quotient(at + unit.at(unit.blocks - 1), share) - c + 1};
        units[{t0, n, h}].push_back({c, b0, b1, slot});
      }
      t0 += n;
    }
  }
  for (auto& [key, total] : blocks) {
    auto [t0, n, h] = key;
    const std::vector<Part>& p = units[key];
    bool ok = !p.empty() && p.front().b0 == 0 && p.back().b1 == total;
    for (size_t i = 0; ok && i < p.size(); ++i) {
      if (i) ok = p[i].b0 == p[i - 1].b1 && p[i].cta == p[0].cta + (int)i && p[i].slot == 2 * p[i].cta;
      else ok = p[0].slot == (p.size() == 1 ? -1 : 2 * p[0].cta + 1);
    }
    if (ok && p.size() > 1) {
      const Join& j = joins[p[0].cta];
      ok = j.t0 == t0 && j.n == n && j.h == h && j.parts == (int)p.size();
    }
    if (!ok) {
      printf("tokens %d .. %d, kv head %d, %d blocks:", t0, t0 + n - 1, h, total);
      for (const Part& x : p) printf(" [%d, %d) by CTA %d", x.b0, x.b1, x.cta);
      printf("\n");
    }
    units.erase(key);
  }
  for (auto& [key, p] : units)
    if (!p.empty()) printf("tokens from %d on, kv head %d: no tile begins or ends so\n", std::get<0>(key), std::get<2>(key));
  for (int c = 0; c < ctas; ++c) {
    const Join& j = joins[c];
    if (j.parts && (j.parts < 2 || c + j.parts > ctas || !blocks.count({j.t0, j.n, j.h}))) printf("CTA %d joins %d parts\n", c, j.parts);
  }
  return 0;
}
