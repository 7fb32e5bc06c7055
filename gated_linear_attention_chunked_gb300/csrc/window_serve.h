// window_serve.h -- launch interface of serving over the windowed attention's pages: packed tokens
// into pages of 16 or 8 bits, pages read back, a token or a chunk of tokens over them.
#pragma once
#include "window_attn.h"

namespace gla {

// The pages of a call (WindowCache): with `exps` their rows are codes of 8 bits, c 2^e, and
// exps [n_pages, pool_layers, KV, slots, 2] holds the exponents of a slot's key and value.
struct ServeCache {
  WindowCache c;      // c.type: the type of the call's keys and values
  signed char* exps = nullptr;
};
// n sequences of tokens packed one behind the other: sequence b's are start[b] .. start[b+1] - 1 of
// n_tokens rows, the first of them at position pos[b].
struct Packed {
  const int* pos;
  const int* start;
  int n_tokens;
};
struct AppendArgs {
  ServeCache cache;
  Packed tok;
  const int* count;  // [n] or null (all): tokens of each sequence that go into its page
  const void* k;     // [n_tokens,KV,96]
  const void* v;     // [n_tokens,KV,192]
};
cudaError_t launch_window_append(const AppendArgs& a, DevCtl ctl, cudaStream_t stream);
// The pages of c.page as 16-bit rows: k [n,slots,KV,96], v [n,slots,KV,192] of type c.type.  pos [n] or null:
// only slots that hold a token of a sequence of so many; copies [n] or null (written): n, or -1 where the page
// is out of range.
cudaError_t launch_window_read8(const ServeCache& cache, void* k, void* v, const int* pos, int* copies,
                                DevCtl ctl, cudaStream_t stream);

struct Decode8Args {
  ServeCache cache;
  const int* pos;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  gla_dtype out_type;
  int H;
  void* workspace;
};
size_t window_decode8_workspace_bytes(int n, int KV, int H, int slots, int n_sm);
cudaError_t launch_window_decode8(const Decode8Args& a, int n_sm, DevCtl ctl, cudaStream_t stream);

struct ChunkArgs {
  ServeCache cache;
  Packed tok;
  const void* q;  // [n_tokens,H,96]
  const void* k;
  const void* v;
  void* o;        // [n_tokens,H,192]
  gla_dtype out_type;
  int H;
  void* workspace;
};
// The same over 8-bit pages where sequences have a few rows (token, query head) each (window_decode8.cu).
size_t window_short8_workspace_bytes(int n, int n_tokens, int KV, int H, int slots, int n_sm);
cudaError_t launch_window_short8(const ChunkArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream);
constexpr int kChunkMostHeads = 128;  // query heads on a key head
size_t window_chunk_workspace_bytes(int n, int n_tokens, int KV, int H, int window, int sink,
                                    bool codes, int n_sm);
cudaError_t launch_window_chunk(const ChunkArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream);

}  // namespace gla
