// emulate FROM TO STALL: cases of the seeds [FROM, TO) of the instances below; STALL 1: one
// completion in each CTA comes so late that waits run out and the kernel ends by itself.
#include <unistd.h>

#include "kernel.h"

using namespace sv;

static std::function<void()> entry;
static std::vector<std::vector<char>> stacks;

static void start() {
  entry();
  cur->done = true;
  swapcontext(&cur->context, &scheduler);
}

// Memory between two pages that cannot be touched; it ends at the upper one.
static void* guarded(size_t bytes) {
  const size_t page = sysconf(_SC_PAGESIZE), n = (bytes + page - 1) / page * page;
  char* p = static_cast<char*>(mmap(nullptr, n + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
  mprotect(p + page, n, PROT_READ | PROT_WRITE);
  return p + page + (n - bytes);
}

static void run_cta(int c, int ctas, int threads, std::function<void()> kernel) {
  blockIdx.x = c;
  gridDim.x = ctas;
  blockDim.x = threads;
  entry = kernel;
  events.clear();
  mbarriers.clear();
  written.clear();
  now_ns = 1000;
  last_product = 0;
  products = copies = 0;
  std::fill(std::begin(async_loads), std::end(async_loads), 0);
  tmem_live = false;
  tmem_base = rng() % 2 * 256;
  for (Barrier& b : barriers) b = Barrier();
  for (Collective& x : collectives) x = Collective();
  for (size_t i = 0; i < shared_bytes; ++i) shared[i] = uint8_t(rng());
  fibers.assign(threads, Fiber());
  stacks.resize(threads);
  for (int i = 0; i < threads; ++i) {
    Fiber& f = fibers[i];
    f.id = i;
    stacks[i].resize(128 << 10);
    getcontext(&f.context);
    f.context.uc_stack.ss_sp = stacks[i].data();
    f.context.uc_stack.ss_size = stacks[i].size();
    f.context.uc_link = nullptr;
    makecontext(&f.context, start, 0);
  }
  // a warp has a speed, which changes at times
  std::vector<int> slow(threads / 32, 1);
  int left = threads;
  for (uint64_t round = 0; left; ++round) {
    if (round % 64 == 0)
      for (int& x : slow) x = 1 + rng() % 8;
    bool any = false;
    for (size_t e = 0; e < events.size();) {
      if (events[e].t > now_ns) {
        ++e;
        continue;
      }
      auto f = events[e].f;
      events[e] = events.back();
      events.pop_back();
      f();
      any = true;
    }
    const int first = rng() % slow.size();
    for (size_t k = 0; k < slow.size(); ++k) {
      const int w = (first + k) % slow.size();
      if (round % slow[w]) continue;
      for (int l = 0; l < 32; ++l) {
        Fiber& f = fibers[w * 32 + l];
        if (f.done || (f.ready && !f.ready())) continue;
        cur = &f;
        swapcontext(&scheduler, &f.context);
        any = true;
        left -= f.done;
      }
    }
    cur = nullptr;
    now_ns += any ? 50 : 200;
    if (now_ns > 10000000000ull) {
      for (Fiber& f : fibers)
        if (!f.done) printf("thread %d waits at %s, line %d\n", f.id, f.where, f.line);
      fail("threads that wait for ever");
    }
  }
  if (tmem_live) fail("TMEM not freed");
  if (products) fail("products in flight at the exit");
  if (copies) fail("copies in flight at the exit");
  for (int n : async_loads)
    if (n) fail("loads in flight at the exit");
}

template <int NR, int D>
void test(int seed, int T, int G, bool stall) {
  using S = TcShape<NR, D>;
  printf("seed %d, %d rows x %d, %d slots\n", seed, NR, D, S::kSlots);
  fflush(stdout);
  rng.seed(seed);
  kWaitNs = stall ? 300000 : 2000000000;
  const bool many = rng() % 3 == 0;
  const int rows = many ? 40 : 1 + rng() % 8, longest = many ? 300 : 1 + rng() % 3000;
  const int H = 2, bs = 16, MB = (longest + T) / bs + 1, NB = 64, ctas = 16;
  AttnArgs a{};
  const size_t nq = size_t(rows) * T * H * G * D;
  auto* bt = static_cast<int32_t*>(guarded(rows * MB * 4));
  auto* sl = static_cast<int32_t*>(guarded(rows * 4));
  auto* scales = static_cast<float*>(guarded(NB * 2 * H * 4));
  int32_t err = 0;
  for (int i = 0; i < rows * MB; ++i) bt[i] = rng() % NB;
  for (int i = 0; i < rows; ++i) sl[i] = rng() % (longest + 1);
  for (int i = 0; i < NB * 2 * H; ++i) scales[i] = 0.01f;
  a.q = guarded(nq * 2);
  a.out = guarded(nq * 2);
  a.scales = scales;
  a.bt = bt;
  a.sl = sl;
  a.scale_log2 = 0.1f;
  a.window = rng() % 4 ? 0 : 1 + rng() % 600;
  a.sinks = a.window ? 4 : 0;
  a.NB = NB;
  a.H = H;
  a.G = G;
  a.D = D;
  a.bs = bs;
  a.B = rows;
  a.T = T;
  a.MB = MB;
  a.block_scales = 2 * H;
  a.R = T * G;
  a.rows_per_block = a.R;
  a.RB = 1;
  a.parts = static_cast<float*>(guarded(size_t(2) * ctas * a.R * D * 4));
  a.stats = static_cast<float2*>(guarded(2 * ctas * a.R * 8));
  a.joins = static_cast<int4*>(guarded(ctas * 16));
  a.err = &err;
  a.wait_ns = kWaitNs;
  a.stall_row = -1;
  a.planes_per_block = 2 * H;
  box_bytes = bs * D;
  shared_bytes = S::kBytes;
  shared = static_cast<uint8_t*>(guarded((shared_bytes + 1023) / 1024 * 1024));
  const int kind = rng() % 3;
  score = [kind]() -> float {
    return kind == 0 ? 0.0f : kind == 1 ? float(int(rng() % 2001) - 1000) : __uint_as_float(rng());
  };
  for (int c = rng() % 4; c < ctas; c += 4) {
    stalling = stall;
    late_in = rng() % 2000;
    run_cta(c, ctas, S::kThreads, [&] { attn_tc_kernel<NR, D>(a, CUtensorMap{}); });
  }
  if (!stall && err) fail("a wait ran out");
}

int main(int, char** argv) {
  const bool stall = atoi(argv[3]);
  for (int seed = atoi(argv[1]); seed < atoi(argv[2]); ++seed) {
    test<24, 128>(seed, 5, 4, stall);
    test<48, 128>(seed, 12, 4, stall);
    test<64, 128>(seed, 16, 4, stall);
    test<24, 64>(seed, 5, 4, stall);
  }
  printf("done\n");
}
