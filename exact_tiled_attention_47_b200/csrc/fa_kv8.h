// fa_kv8.h -- launchers of the paged 8-bit cache (append, attention) and of the page operations,
// shared between their C-ABI layer (fa_kv8_api.cu) and the kernel files.  Arguments reaching these
// functions have already been validated.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace fa {

constexpr int kKv8Block = 16;  // tokens of one head that share a scale

// The pools of a paged 8-bit cache and how sequences map to them.  A page holds, head after head, its
// page_size rows of D codes: row r of head h of page p starts at ((p * Hkv + h) * page_size + r) * D,
// its scale is at (p * Hkv + h) * (page_size / 16) + r / 16.
struct Kv8Cache {
  void* k;
  void* v;
  float* ks;
  float* vs;
  const int* table;    // [B, pages_per_seq]
  const int* seqlens;  // [B] (attention: nullptr = the whole table is in use)
  int B, Hkv, D, num_pages, page_size, pages_per_seq;
  int int8;  // codes: 1 = int8, 0 = e4m3
};

struct AppendArgs {
  Kv8Cache c;
  const void* k;  // new rows [B, Nt, Hkv, D], fp16 or bf16
  const void* v;
  const int* new_lens;  // [B] or nullptr (all Nt)
  int Nt, fp16;
  int* status;
};

struct Attend8Args {
  Kv8Cache c;
  const void* q;  // [B, Nq, Hq, D]
  void* o;
  float* lse;  // [B, Hq, Nq]
  void* ws;
  int Nq, Hq;
  float scale;
  int fp16, o_fp32;
  int* status;
};

// Page pools by value in a kernel's parameters; more pools than this take several launches.
constexpr int kMaxPools = 64;
struct PoolSet {
  const void* src[kMaxPools];
  void* dst[kMaxPools];
  unsigned long long page_bytes[kMaxPools];
  int n;
};

struct PagesArgs {
  int* table;    // [S, pages_per_seq]
  int* seqlens;  // [S]
  int* refs;     // [num_pages]
  const int* a;  // slots (extend, free), sources (fork, copy)
  const int* b;  // lengths to add (extend), destinations (fork, copy)
  int n, S, pages_per_seq, num_pages, page_size;
  int dst_pages;  // copy: pages of the destination pools
  int* table_out;  // compact
  int* refs_out;
  int* remap;
  int* n_live;
  const void* const* src_pools;
  void* const* pools;
  const size_t* page_bytes;
  int n_pools;
  int* ws;
  int* status;
};

size_t kv8_chunk_ws_bytes(int D);
size_t kv8_attend_ws_bytes(int B, int Nq, int Hq, int Hkv, int D);
size_t pages_ws_bytes(int n, int S, int num_pages);

// Return a cudaError_t-compatible code (0 = success).
int launch_kv8_append(const AppendArgs& a, cudaStream_t stream);
int launch_kv8_chunk(const Attend8Args& a, cudaStream_t stream);  // many rows per KV head
int launch_kv8_attend(const Attend8Args& a, cudaStream_t stream);
int launch_pages_extend(const PagesArgs& a, cudaStream_t stream);
int launch_pages_free(const PagesArgs& a, cudaStream_t stream);
int launch_pages_fork(const PagesArgs& a, cudaStream_t stream);
int launch_pages_compact(const PagesArgs& a, cudaStream_t stream);
int launch_pages_copy(const PagesArgs& a, cudaStream_t stream);

}  // namespace fa
