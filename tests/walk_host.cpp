// Runs the walk of attention's workgroups over their shares on the host: a thread
// for each lane, barriers for the workgroup's and for a wave's exchanges, and waves
// that come out of every barrier late.  Checks that all lanes of a workgroup have
// one place throughout, and that the shares have every key of every tile once.
#include <pthread.h>
#include <unistd.h>

#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <thread>
#include <tuple>
#include <vector>

#include "acp_attn.hpp"
#include "acp_engine.hpp"

namespace {
struct Index {
  uint32_t x;
};
thread_local Index threadIdx;
pthread_barrier_t g_all, g_wave[8];
unsigned long long g_slots[8][64];
int g_late;  // 1: all waves but the first, 2: the first

void __syncthreads() {
  pthread_barrier_wait(&g_all);
  const bool first = threadIdx.x < 64;
  if ((g_late == 1 && !first) || (g_late == 2 && first)) usleep(4000);
}
unsigned long long __shfl_up(unsigned long long v, uint32_t d) {
  const uint32_t w = threadIdx.x / 64, lane = threadIdx.x % 64;
  g_slots[w][lane] = v;
  pthread_barrier_wait(&g_wave[w]);
  const unsigned long long r = lane >= d ? g_slots[w][lane - d] : v;
  pthread_barrier_wait(&g_wave[w]);
  return r;
}
int __builtin_amdgcn_readfirstlane(int v) { return v; }  // of values that all lanes hold
uint64_t __builtin_amdgcn_ballot_w64(bool) { abort(); }  // not on the walk's way
}  // namespace

namespace acp {
namespace dev {
inline uint32_t divide(uint32_t n, const Div& d) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.mag) >> (31 + d.sh));
}
}  // namespace dev
}  // namespace acp

#include "acp_dev_walk.hpp"

namespace {

using Step = std::tuple<uint32_t, uint32_t, uint32_t, uint32_t, bool, bool, uint32_t>;  // seq, tile, keys [,), head, tail, meets

template <int M, uint32_t CUT, uint32_t LANES>
std::vector<std::vector<Step>> workgroup(const acp::AttendArgs& A, uint32_t index) {
  static uint64_t space[acp::dev::kWalkWords];
  std::vector<std::vector<Step>> steps(LANES);
  pthread_barrier_init(&g_all, nullptr, LANES);
  for (uint32_t w = 0; w < LANES / 64; ++w) pthread_barrier_init(&g_wave[w], nullptr, 64);
  std::vector<std::thread> lanes;
  for (uint32_t l = 0; l < LANES; ++l)
    lanes.emplace_back([&, l] {
      threadIdx.x = l;
      acp::dev::Walk<M, CUT, true> walk;
      if (!walk.begin_at(A, index, space)) return;
      bool more;
      do {
        acp::dev::Tile t;
        if (walk.seq >= A.batch.sequences || !t.template set<M>(A, walk.seq, walk.tile)) {
          std::printf("lane %u of workgroup %u has tile %u of sequence %u\n", l, index, walk.tile, walk.seq);
          std::fflush(stdout);
          _exit(1);
        }
        walk.cut(A, static_cast<uint32_t>(t.keys));
        steps[l].push_back({walk.seq, walk.tile, walk.begin, walk.end, walk.head, walk.tail, walk.tail ? 1u : walk.meets(A)});
        walk.put(space);
        __syncthreads();
        walk.take(space);
        more = walk.next(A);
        __syncthreads();
      } while (more);
    });
  for (auto& t : lanes) t.join();
  pthread_barrier_destroy(&g_all);
  for (uint32_t w = 0; w < LANES / 64; ++w) pthread_barrier_destroy(&g_wave[w]);
  return steps;
}

template <int M, uint32_t CUT, uint32_t LANES>
int batch(std::mt19937& rng, int sequences, int most_new, int most_length, uint32_t group, uint32_t shares) {
  std::vector<int32_t> starts(1, 0), lengths;
  for (int s = 0; s < sequences; ++s) {
    const int n = static_cast<int>(rng() % (most_new + 1));
    starts.push_back(starts.back() + n);
    lengths.push_back(n == 0 ? static_cast<int>(rng() % 5) : n + static_cast<int>(rng() % most_length));
  }
  acp::AttendArgs A{};
  auto div = [](uint32_t d) {
    acp::Div r{d, 0, 0};
    acp::magic_for(d, &r.mag, &r.sh);
    return r;
  };
  A.batch.starts = starts.data();
  A.batch.lengths = lengths.data();
  A.batch.sequences = static_cast<uint32_t>(sequences);
  A.batch.page = div(16);
  A.batch.max_pages = static_cast<uint32_t>((most_new + most_length) / 16 + 1);
  A.group = div(group);
  A.kv_heads = div(1);
  A.tokens = static_cast<uint32_t>(starts.back());
  A.shares = shares;
  A.least = 256;
  std::map<std::pair<uint32_t, uint32_t>, std::map<uint32_t, Step>> tiles;  // by the share's first place: begin
  std::map<std::pair<uint32_t, uint32_t>, int> parts;
  for (uint32_t w = 0; w < shares; ++w) {
    const auto steps = workgroup<M, CUT, LANES>(A, w);
    for (uint32_t l = 1; l < LANES; ++l)
      if (steps[l] != steps[0]) return std::printf("lane %u of workgroup %u went another way\n", l, w), 1;
    for (const Step& s : steps[0]) {
      const auto key = std::make_pair(std::get<0>(s), std::get<1>(s));
      ++parts[key];
      if (std::get<2>(s) < std::get<3>(s) && !tiles[key].insert({std::get<2>(s), s}).second)
        return std::printf("keys twice\n"), 1;
      if (std::get<4>(s) && std::get<2>(s) != 0) return std::printf("a head that begins late\n"), 1;
    }
    for (const Step& s : steps[0])
      if (std::get<4>(s)) parts[{std::get<0>(s), std::get<1>(s)}] -= static_cast<int>(std::get<6>(s));
  }
  uint64_t keys = 0;
  for (int s = 0; s < sequences; ++s) {
    const int n = starts[s + 1] - starts[s];
    const uint32_t rows = static_cast<uint32_t>(n) * group;
    for (uint32_t i = 0; i * M < rows; ++i) {
      const uint32_t last = std::min<uint32_t>(rows, (i + 1) * M) - 1;
      const uint32_t want = static_cast<uint32_t>(lengths[s] - n) + last / group + 1;
      uint32_t at = 0;
      for (const auto& p : tiles[{s, i}]) {
        if (p.first != at) return std::printf("a gap before key %u\n", p.first), 1;
        at = std::get<3>(p.second);
      }
      if (at != want) return std::printf("tile %u of sequence %d ends at %u and not %u\n", i, s, at, want), 1;
      if (parts[{s, i}] != 0) return std::printf("a tile's number of shares is wrong\n"), 1;
      keys += want;
    }
  }
  std::printf("%d sequences, %llu keys, %u shares\n", sequences, static_cast<unsigned long long>(keys), shares);
  std::fflush(stdout);
  return 0;
}

}  // namespace

int main() {
  std::mt19937 rng(7);
  for (g_late = 0; g_late < 3; ++g_late) {
    const int rounds = g_late ? 1 : 2;
    for (int k = 0; k < rounds; ++k) {
      if (batch<16, acp::kCutStep, 256>(rng, 3, 1, 3000, 4, 7)) return 1;
      if (batch<16, acp::kCutStep, 256>(rng, 40, 3, 300, 3, 5)) return 1;
      if (batch<16, acp::kCutStep, 256>(rng, 300, 1, 40, 8, 3)) return 1;
      if (batch<256, acp::kCutPrompt, 512>(rng, 5, 200, 1500, 2, 6)) return 1;
      if (batch<128, acp::kCutPrompt, 256>(rng, 2, 90, 4000, 5, 9)) return 1;
    }
  }
  std::printf("ok\n");
  return 0;
}
