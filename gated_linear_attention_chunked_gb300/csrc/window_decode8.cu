// window_decode8.cu -- the decode step and short chunks over pages of 8 bits (window_rows8.cuh).
#include "window_rows8.cuh"

namespace gla {
namespace {

// Units have 8, 16, 24 or 32 rows: as many as a sequence has, since each unit of its own turns the page's codes
// into operands again.
int unit_rows(long long rows) { return rows >= 25 ? 32 : rows >= 17 ? 24 : rows >= 9 ? 16 : 8; }

rows8::Plan decode_plan(int n, int KV, int H, int slots, int n_sm) {
  const int G = H / KV, rows = unit_rows(G);
  const long long units = (long long)n * KV * ((G + rows - 1) / rows);
  return rows8::make_plan(units, units, rows, slots, n_sm);
}
// Units of packed tokens: how the rows fall into sequences only the device knows.
rows8::Plan short_plan(int n, int n_tokens, int KV, int H, int slots, int n_sm) {
  const int some = std::min(n, n_tokens);
  const long long each = (long long)((n_tokens + some - 1) / some) * (H / KV);  // rows
  const int rows = unit_rows(each);
  const long long most = ((long long)n_tokens * (H / KV) / rows + some) * KV;
  return rows8::make_plan(most, std::min(some * ((each + rows - 1) / rows) * KV, most), rows, slots, n_sm);
}

}  // namespace

size_t window_decode8_workspace_bytes(int n, int KV, int H, int slots, int n_sm) {
  return rows8::workspace_bytes(decode_plan(n, KV, H, slots, n_sm));
}

cudaError_t launch_window_decode8(const Decode8Args& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const WindowCache& c = a.cache.c;
  const rows8::Args r{a.cache, {a.pos, nullptr, c.n}, a.q, a.k, a.v, a.o, a.H, a.workspace};
  return rows8::launch(r, a.out_type, decode_plan(c.n, c.KV, a.H, c.window + c.sink, n_sm), ctl, stream);
}

size_t window_short8_workspace_bytes(int n, int n_tokens, int KV, int H, int slots, int n_sm) {
  return rows8::workspace_bytes(short_plan(n, n_tokens, KV, H, slots, n_sm));
}

cudaError_t launch_window_short8(const ChunkArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const WindowCache& c = a.cache.c;
  const rows8::Args r{a.cache, a.tok, a.q, a.k, a.v, a.o, a.H, a.workspace};
  return rows8::launch(r, a.out_type,
                       short_plan(c.n, a.tok.n_tokens, c.KV, a.H, c.window + c.sink, n_sm), ctl, stream);
}

}  // namespace gla
