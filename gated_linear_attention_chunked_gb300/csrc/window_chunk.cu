// window_chunk.cu -- chunks of new tokens over pages of 16 bits, the cut of items into parts and their
// join (window_chunk.cuh).
#include "window_chunk.cuh"

namespace gla {
namespace {

using namespace chunk;

// Items are cut where whole ones leave SMs without work: into the parts whose rounds over the device take
// least, counting a tile of keys as 1, what an item needs besides its tiles as 2, and a part's results,
// written and joined, as 2; and of those within a 32nd of the least into the fewest, since each part takes 776 bytes of
// workspace a (token, query head), so that a gain below the model's own error costs none.  How many items there are,
// and how many tiles each has, only the device knows: the sequences are taken for equally long and their windows for
// full.
Plan make_plan(int n, int n_tokens, int KV, int H, int window, int sink, int n_sm) {
  Plan p;
  const int G = H / KV;
  p.per = BM / G;
  n_sm = std::max(n_sm, 1);
  p.units = ((long long)n_tokens / p.per + std::min(n, n_tokens)) * KV;
  const long long tokens = (n_tokens + n - 1) / n;  // of a sequence
  const long long items = std::max(1ll, n_tokens / tokens) * ((tokens + p.per - 1) / p.per) * KV;
  const double tiles = (window + (double)sink + p.per) / BN + 1.5;
  auto cost = [&](int parts) {
    const double rounds = (double)((items * parts + n_sm - 1) / n_sm);
    return rounds * (tiles / parts + 2 + (parts > 1 ? 2 : 0)) + (parts > 1 ? 2 : 0);
  };
  const int most = std::min(kMostParts, std::max((int)((tiles + 1) / 2), 1));
  double best = cost(1);
  for (int parts = 2; parts <= most; ++parts) best = std::min(best, cost(parts));
  p.parts = 1;
  while (cost(p.parts) > best * (33.0 / 32)) ++p.parts;
  const long long all = p.units * p.parts;
  // a CTA an SM, and more where its list of items would not hold them
  p.grid = (unsigned)std::max(std::min<long long>(all, n_sm), (all + LIST - 1) / LIST);
  const size_t rows = (size_t)n_tokens * H * p.parts;
  p.ml = ((p.units + 1) * 8 + 255) / 256 * 256;
  p.o = p.ml + (rows * 8 + 255) / 256 * 256;
  p.bytes = p.parts > 1 ? p.o + rows * kDV * 4 : 0;
  return p;
}

// Over pages of 8 bits, sequences of a few rows each go to warp-level products (window_rows8.cuh), which
// turn a code into an operand in registers; here it goes through shared memory, and a tile of 128 rows is
// mostly empty.
bool is_short(int n, int n_tokens, int KV, int H) {
  return (long long)n_tokens * (H / KV) <= 32ll * std::min(n, n_tokens);
}

// Over pages of 8 bits, where sequences have more than two items of 128 rows each, the pages are first written
// out as 16-bit rows, each once: an item that turns a tile of codes into operands for itself takes 2.8 us
// for it (four warps do), one over 16 bits 1.2, and the copy costs HBM 864 bytes a slot and key head.  4 x 2,048
// tokens of 16 heads on 1,024 slots of 4 key heads: 102 us in place of 145; with two items each 96 x 64 tokens on
// 2,052 slots 261 in place of 276, 60 tokens on 16,388 37 in place of 36; with one 96 x 32 tokens 219 in place
// of 152.  As long as the copy stays below a GiB.
struct Copy {
  size_t v, pages, bytes;  // offsets of the values and of the copies' indexes; a multiple of 256
};
bool copies_pages(int n, int n_tokens, int KV, int H, int window, int sink, Copy* copy) {
  const size_t rows = (size_t)n * (window + (size_t)sink) * KV;
  if ((long long)n_tokens * (H / KV) <= 256ll * n || rows > (1u << 30) / (2 * (kDK + kDV))) return false;
  copy->v = (rows * kDK * 2 + 255) / 256 * 256;
  copy->pages = copy->v + (rows * kDV * 2 + 255) / 256 * 256;
  copy->bytes = copy->pages + ((size_t)n * 4 + 255) / 256 * 256;
  return true;
}

template <class TO>
cudaError_t join(const ChunkArgs& a, const Plan& plan, cudaStream_t stream) {
  const int rows = plan.per * (a.H / a.cache.c.KV);
  PdlLaunch l(dim3((unsigned)plan.units, (unsigned)rows), dim3(JOIN_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&l.cfg, window_chunk_join_kernel<TO>, a, plan);
}

}  // namespace

size_t window_chunk_workspace_bytes(int n, int n_tokens, int KV, int H, int window, int sink,
                                    bool codes, int n_sm) {
  if (codes && is_short(n, n_tokens, KV, H))
    return window_short8_workspace_bytes(n, n_tokens, KV, H, window + sink, n_sm);
  const Plan p = make_plan(n, n_tokens, KV, H, window, sink, n_sm);
  Copy copy;
  const size_t pages = codes && copies_pages(n, n_tokens, KV, H, window, sink, &copy) ? copy.bytes : 0;
  return pages + p.bytes;
}

cudaError_t launch_window_chunk(const ChunkArgs& call, int n_sm, DevCtl ctl, cudaStream_t stream) {
  ChunkArgs a = call;
  WindowCache& c = a.cache.c;
  if (a.cache.exps && is_short(c.n, a.tok.n_tokens, c.KV, a.H))
    return launch_window_short8(a, n_sm, ctl, stream);
  const Plan plan = make_plan(c.n, a.tok.n_tokens, c.KV, a.H, c.window, c.sink, n_sm);
  cudaError_t e;
  Copy copy;
  if (a.cache.exps && copies_pages(c.n, a.tok.n_tokens, c.KV, a.H, c.window, c.sink, &copy)) {
    char* const to = static_cast<char*>(a.workspace);
    int* const pages = reinterpret_cast<int*>(to + copy.pages);
    if ((e = launch_window_read8(a.cache, to, to + copy.v, a.tok.pos, pages, ctl, stream)) != cudaSuccess) return e;
    c.k = to;
    c.v = to + copy.v;
    c.page = pages;
    c.n_pages = c.n;
    c.pool_layers = 1;
    c.layer = 0;
    a.cache.exps = nullptr;
    a.workspace = to + copy.bytes;
  }
  if (a.cache.exps) e = launch8(a, plan, ctl, stream);
  else if (c.type == GLA_BF16) e = run<__nv_bfloat16, false>(a, plan, ctl, stream);
  else e = run<__half, false>(a, plan, ctl, stream);
  if (e != cudaSuccess || plan.parts == 1) return e;
  if (a.out_type == GLA_FP32) return join<float>(a, plan, stream);
  return a.out_type == GLA_BF16 ? join<__nv_bfloat16>(a, plan, stream) : join<__half>(a, plan, stream);
}

}  // namespace gla
