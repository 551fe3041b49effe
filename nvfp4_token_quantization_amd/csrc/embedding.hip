// embedding.hip -- rows of a table by token id, scaled, and the table's
// gradient by sorted tokens (gfx950).
//
//   out[i] = scale table[ids[i]]
//   dtable[v] = add[v] + scale sum over the tokens i with ids[i] = v of dout[i]
//
// HBM-bound both ways.  Forward: one wave per 512 columns of a token.
//
// Backward, nothing by atomics, a row's tokens added in the order of the tokens:
//  1. embed_rank_kernel sorts chunks of 2048 ids by counting: an id's place in
//     its chunk is the number of ids below it and of equal ids before it.
//  2. embed_merge_kernel (more than one chunk): an id's place in the whole is
//     its place in its chunk plus, for every other chunk, the ids there that
//     go before it (a binary search).  Stable, since equal ids of earlier
//     chunks go before and those of later ones do not.
//  3. embed_sum_kernel: a wave adds the rows of EMBED-run consecutive sorted
//     tokens in fp32, 512 columns, and writes a table row when its id's run
//     ends; runs that cross into another wave's tokens leave partial rows.
//     Other blocks of the same launch meanwhile write the table rows that no
//     token names (zeros, or add; nothing when the sum goes in place).
//  4. embed_join_kernel adds the partial rows of a run that crosses.
#include "rowwise.h"

namespace nvfp4 {

constexpr int EMBED_CHUNK = 2048;  // ids sorted together
constexpr int EMBED_RANK = 64;     // ids a block of step 1 places, by 4 slices of the chunk
constexpr int EMBED_MERGE = 128;   // ids a block of step 2 places, by 8 slices of the chunks
constexpr int EMBED_ROWS = 64;     // table rows a block looks for and fills
constexpr uint32_t EMBED_NONE = 0x7FFFFFFFu;  // an id outside the table: sorted last

struct EmbedArgs {
  const int32_t* ids;
  const void* in;   // table (forward) or dout
  const void* add;  // backward, may be NULL
  void* out;
  int64_t tokens, vocab, d;
  float scale;
  bool in_bf, out_bf;
  uint32_t* key[2];  // sorted ids: of the chunks, of all
  int32_t* pos[2];   // their tokens
  int sorted;        // which of the two holds the whole order
  float* part;       // [blocks of a run][2][d]: a block's first run, when it goes on from the block
                     // before, and its last, when it goes on to the next
  int64_t run;       // sorted tokens a wave adds
  int64_t runs;
  int pieces;        // of 512 columns
};

__device__ __forceinline__ uint32_t embed_key(const EmbedArgs& p, int64_t i) {
  const int32_t id = p.ids[i];
  return id >= 0 && id < p.vocab ? (uint32_t)id : EMBED_NONE;
}

template <bool VEC>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t items = p.tokens * p.pieces;
  for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t t = item / p.pieces;
    const int piece = (int)(item % p.pieces);
    const int32_t id = p.ids[t];
    float v[8] = {};
    if (id >= 0 && id < p.vocab) {
      load8<VEC>(row_at(p.in, p.in_bf, id, p.d), p.in_bf, p.d, piece, 64, lane, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= p.scale;
    }
    store8<VEC>(row_at(p.out, p.out_bf, t, p.d), p.out_bf, p.d, piece, 64, lane, v);
  }
}

__global__ __launch_bounds__(256) void embed_rank_kernel(EmbedArgs p) {
  __shared__ __attribute__((aligned(16))) uint32_t s_key[EMBED_CHUNK];
  __shared__ int s_rank[4][EMBED_RANK];
  const int tid = threadIdx.x, lane = tid & 63, slice = tid >> 6;
  constexpr int PARTS = EMBED_CHUNK / EMBED_RANK;
  const int64_t c0 = (int64_t)(blockIdx.x / PARTS) * EMBED_CHUNK;
  const int own = (int)(blockIdx.x % PARTS) * EMBED_RANK + lane;  // within the chunk
  const int n = (int)min((int64_t)EMBED_CHUNK, p.tokens - c0);
  for (int i = tid; i < EMBED_CHUNK; i += 256) s_key[i] = i < n ? embed_key(p, c0 + i) : 0xFFFFFFFFu;  // goes before none
  __syncthreads();
  const uint32_t mine = s_key[own];
  const int per = EMBED_CHUNK / 4;
  int rank = 0;
  const uint4* q = reinterpret_cast<const uint4*>(s_key + slice * per);
#pragma unroll 4
  for (int i = 0; i < per / 4; ++i) {
    const uint4 k = q[i];
    const int at = slice * per + 4 * i;
    // equal ids go before when their token does
    rank += k.x < mine + (at < own);
    rank += k.y < mine + (at + 1 < own);
    rank += k.z < mine + (at + 2 < own);
    rank += k.w < mine + (at + 3 < own);
  }
  s_rank[slice][lane] = rank;
  __syncthreads();
  if (slice == 0 && own < n) {
    const int64_t at = c0 + s_rank[0][lane] + s_rank[1][lane] + s_rank[2][lane] + s_rank[3][lane];
    p.key[0][at] = mine;
    p.pos[0][at] = (int32_t)(c0 + own);
  }
}

__global__ __launch_bounds__(1024) void embed_merge_kernel(EmbedArgs p) {
  __shared__ uint32_t s_key[8][EMBED_CHUNK];
  __shared__ int s_rank[8][EMBED_MERGE];
  const int tid = threadIdx.x, slice = tid / EMBED_MERGE, me = tid % EMBED_MERGE;
  const int64_t i = (int64_t)blockIdx.x * EMBED_MERGE + me;  // place in the chunks' order
  const int64_t chunks = (p.tokens + EMBED_CHUNK - 1) / EMBED_CHUNK, mine = i / EMBED_CHUNK;  // the block's, all of it
  const uint32_t key = i < p.tokens ? p.key[0][i] : 0u;
  int before = 0;
  for (int64_t g = 0; g < chunks; g += 8) {
    const int64_t first = g * EMBED_CHUNK, n = min((int64_t)8 * EMBED_CHUNK, p.tokens - first);
    for (int64_t k = tid; k < n; k += 1024) s_key[k / EMBED_CHUNK][k % EMBED_CHUNK] = p.key[0][first + k];
    __syncthreads();
    const int64_t c = g + slice;
    if (c < chunks && c != mine) {
      // ids of chunk c below the limit go before: equal ones of an earlier chunk too
      const uint32_t limit = key + (c < mine);
      int lo = 0, hi = (int)min((int64_t)EMBED_CHUNK, p.tokens - c * EMBED_CHUNK);
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_key[slice][mid] < limit) lo = mid + 1;
        else hi = mid;
      }
      before += lo;
    }
    __syncthreads();
  }
  s_rank[slice][me] = before;
  __syncthreads();
  if (slice == 0 && i < p.tokens) {
    int64_t at = i - mine * EMBED_CHUNK;
    for (int k = 0; k < 8; ++k) at += s_rank[k][me];
    p.key[1][at] = key;
    p.pos[1][at] = p.pos[0][i];
  }
}

// first place in the sorted ids whose id is not below `id`
__device__ __forceinline__ int64_t embed_lower(const EmbedArgs& p, uint32_t id) {
  const uint32_t* key = p.key[p.sorted];
  int64_t lo = 0, hi = p.tokens;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (key[mid] < id) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// table row v = add[v] + scale * sum
template <bool VEC>
__device__ __forceinline__ void embed_write(const EmbedArgs& p, uint32_t v, int piece, int lane, const float (&sum)[8]) {
  float o[8] = {};
  if (p.add) load8<VEC>(row_at(p.add, p.out_bf, v, p.d), p.out_bf, p.d, piece, 64, lane, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = p.add ? __builtin_fmaf(p.scale, sum[i], o[i]) : p.scale * sum[i];
  store8<VEC>(row_at(p.out, p.out_bf, v, p.d), p.out_bf, p.d, piece, 64, lane, o);
}

constexpr int EMBED_AHEAD = 8;  // rows in flight

template <bool VEC>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedArgs p, int64_t sum_blocks) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (blockIdx.x >= sum_blocks) {
    // table rows that no token names
    const int64_t v0 = (int64_t)(blockIdx.x - sum_blocks) * EMBED_ROWS, v = v0 + lane;
    const int64_t at = v < p.vocab ? embed_lower(p, (uint32_t)v) : p.tokens;
    const bool named = v >= p.vocab || (at < p.tokens && p.key[p.sorted][at] == (uint32_t)v);
    uint64_t fill = ~__ballot(named);
    while (fill) {
      const int r = __builtin_ctzll(fill);
      fill &= fill - 1;
      for (int piece = tid >> 6; piece < p.pieces; piece += 4) {
        float o[8] = {};
        if (p.add) load8<VEC>(row_at(p.add, p.out_bf, v0 + r, p.d), p.out_bf, p.d, piece, 64, lane, o);
        store8<VEC>(row_at(p.out, p.out_bf, v0 + r, p.d), p.out_bf, p.d, piece, 64, lane, o);
      }
    }
    return;
  }
  const int64_t item = (int64_t)blockIdx.x * 4 + (tid >> 6);
  const int64_t b = item / p.pieces;
  const int piece = (int)(item % p.pieces);
  if (b >= p.runs) return;
  const uint32_t* key = p.key[p.sorted];
  const int32_t* pos = p.pos[p.sorted];
  const int64_t i0 = b * p.run, i1 = min(p.tokens, i0 + p.run);
  const int n = (int)(i1 - i0);  // at most 64
  const uint32_t my_key = lane < n ? key[i0 + lane] : EMBED_NONE;
  const int32_t my_pos = lane < n ? pos[i0 + lane] : 0;
  const uint32_t prev = i0 > 0 ? key[i0 - 1] : EMBED_NONE, next = i1 < p.tokens ? key[i1] : EMBED_NONE;
  const uint64_t live = __ballot(my_key != EMBED_NONE);  // the first `count` lanes
  const int count = __popcll(live);
  float sum[8] = {};
  for (int g = 0; g < count; g += EMBED_AHEAD) {
    float v[EMBED_AHEAD][8];
#pragma unroll
    for (int k = 0; k < EMBED_AHEAD; ++k)
      if (g + k < count) {
        const int32_t t = __builtin_amdgcn_readlane(my_pos, g + k);
        load8<VEC>(row_at(p.in, p.in_bf, t, p.d), p.in_bf, p.d, piece, 64, lane, v[k]);
      }
#pragma unroll
    for (int k = 0; k < EMBED_AHEAD; ++k) {
      if (g + k >= count) break;
      const int i = g + k;
      const uint32_t id = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[k][e];
      const uint32_t after = i + 1 < n ? (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 1) : next;
      if (after == id && i + 1 < n) continue;
      // the id's run ends here, or goes on past this wave's tokens
      const bool from_before = id == prev, goes_on = after == id;
      if (from_before || goes_on)
        store8<VEC>(p.part + (2 * b + (from_before ? 0 : 1)) * p.d, false, p.d, piece, 64, lane, sum);
      else
        embed_write<VEC>(p, id, piece, lane, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    }
  }
}

// Block (b, piece): the run that starts in b's tokens and goes on past them.
constexpr int EMBED_JOIN = 8;  // waves that share the partial rows
template <bool VEC>
__global__ __launch_bounds__(64 * EMBED_JOIN) void embed_join_kernel(EmbedArgs p) {
  __shared__ float s_sum[EMBED_JOIN][8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b = blockIdx.x / p.pieces;
  const int piece = (int)(blockIdx.x % p.pieces);
  const uint32_t* key = p.key[p.sorted];
  const int64_t i0 = b * p.run, i1 = i0 + p.run;  // i1 <= tokens: the last block is not launched
  const uint32_t id = key[i1 - 1];
  if (id == EMBED_NONE || key[i1] != id || (i0 > 0 && key[i0 - 1] == id)) return;  // block-uniform
  const int64_t last = (embed_lower(p, id + 1) - 1) / p.run;  // block of its last token
  float sum[8] = {};
  if (wave == 0) load8<VEC>(p.part + (2 * b + 1) * p.d, false, p.d, piece, 64, lane, sum);
  const int64_t rows = last - b, per = (rows + EMBED_JOIN - 1) / EMBED_JOIN, end = min(rows, (wave + 1) * per);
#pragma unroll 4
  for (int64_t k = wave * per; k < end; ++k) {
    float v[8];
    load8<VEC>(p.part + 2 * (b + 1 + k) * p.d, false, p.d, piece, 64, lane, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += v[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s_sum[wave][e][lane] = sum[e];
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < EMBED_JOIN; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += s_sum[w][e][lane];
  embed_write<VEC>(p, id, piece, lane, sum);
}

static bool embed_vec(int64_t d, const void* a, const void* b, const void* c) {
  return d % 8 == 0 && nvfp4host::aligned(a, 16) && nvfp4host::aligned(b, 16) && nvfp4host::aligned(c, 16);
}

// Sorted tokens a wave adds: 64 at most (its lanes hold their ids), and fewer
// where that leaves CUs without a wave.
static int64_t embed_run(int64_t tokens, int64_t pieces) {
  int64_t run = 64;
  while (run > 8 && tokens * pieces < run * 4 * 256) run /= 2;
  return run;
}

static int64_t embed_bytes(int64_t tokens, int64_t d) {
  const int64_t pieces = (d + 511) / 512, run = embed_run(tokens, pieces);
  const int64_t runs = (tokens + run - 1) / run, lists = (tokens + 3) / 4 * 4;
  return 4 * 4 * lists + (runs > 1 ? runs * 2 * d * 4 : 0);
}

}  // namespace nvfp4

using nvfp4host::aligned;

static bool bad_type(int t) { return t != NVFP4_TYPE_F32 && t != NVFP4_TYPE_BF16; }
static bool bad_elem(const void* p, int t) { return !aligned(p, t == NVFP4_TYPE_BF16 ? 2 : 4); }

static int embed_sizes(int64_t tokens, int64_t vocab, int64_t d) {
  if (tokens < 0 || vocab < 0 || d < 0) return NVFP4_ERROR_INVALID_VALUE;
  if (tokens > ((int64_t)1 << 24) || vocab >= ((int64_t)1 << 31) - 1 || d > ((int64_t)1 << 20))
    return NVFP4_ERROR_UNSUPPORTED_SHAPE;
  return NVFP4_SUCCESS;
}

extern "C" int nvfp4_embedding(const void* table, int table_type, int64_t vocab, const int32_t* ids, int64_t tokens,
                               int64_t d, float scale, void* out, int out_type, void* stream) {
  if (bad_type(table_type) || bad_type(out_type)) return NVFP4_ERROR_INVALID_VALUE;
  int st = embed_sizes(tokens, vocab, d);
  if (st) return st;
  if (tokens == 0 || d == 0) return NVFP4_SUCCESS;
  if ((vocab > 0 && !table) || !ids || !out) return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(table, table_type) || bad_elem(out, out_type) || !aligned(ids, 4)) return NVFP4_ERROR_MISALIGNED;
  if ((st = nvfp4host::check_arch())) return st;
  nvfp4::EmbedArgs p{};
  p.ids = ids; p.in = table; p.out = out; p.tokens = tokens; p.vocab = vocab; p.d = d; p.scale = scale;
  p.in_bf = table_type == NVFP4_TYPE_BF16; p.out_bf = out_type == NVFP4_TYPE_BF16;
  p.pieces = (int)((d + 511) / 512);
  const int64_t blocks = (tokens * p.pieces + 3) / 4;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (nvfp4::embed_vec(d, table, out, nullptr))
    hipLaunchKernelGGL(nvfp4::embed_kernel<true>, grid, dim3(256), 0, (hipStream_t)stream, p);
  else
    hipLaunchKernelGGL(nvfp4::embed_kernel<false>, grid, dim3(256), 0, (hipStream_t)stream, p);
  return nvfp4host::launch_status();
}

extern "C" int64_t nvfp4_embedding_backward_workspace(int64_t tokens, int64_t d) {
  return tokens <= 0 || d <= 0 || embed_sizes(tokens, 0, d) ? 0 : nvfp4::embed_bytes(tokens, d);
}

extern "C" int nvfp4_embedding_backward(const void* dout, int dout_type, const int32_t* ids, int64_t tokens,
                                        int64_t vocab, int64_t d, float scale, const void* add, void* dtable,
                                        int dtable_type, void* workspace, int64_t workspace_bytes, void* stream) {
  if (bad_type(dout_type) || bad_type(dtable_type)) return NVFP4_ERROR_INVALID_VALUE;
  int st = embed_sizes(tokens, vocab, d);
  if (st) return st;
  if (vocab == 0 || d == 0) return NVFP4_SUCCESS;
  if (!dtable || (tokens > 0 && (!dout || !ids))) return NVFP4_ERROR_INVALID_VALUE;
  if (workspace_bytes < nvfp4_embedding_backward_workspace(tokens, d) || (tokens > 0 && !workspace))
    return NVFP4_ERROR_INVALID_VALUE;
  if (bad_elem(dout, dout_type) || bad_elem(dtable, dtable_type) || bad_elem(add, dtable_type) || !aligned(ids, 4) ||
      !aligned(workspace, 16))
    return NVFP4_ERROR_MISALIGNED;
  if (tokens == 0 && add == dtable) return NVFP4_SUCCESS;
  if ((st = nvfp4host::check_arch())) return st;
  nvfp4::EmbedArgs p{};
  p.ids = ids; p.in = dout; p.add = add; p.out = dtable; p.tokens = tokens; p.vocab = vocab; p.d = d; p.scale = scale;
  p.in_bf = dout_type == NVFP4_TYPE_BF16; p.out_bf = dtable_type == NVFP4_TYPE_BF16;
  p.pieces = (int)((d + 511) / 512);
  p.run = nvfp4::embed_run(tokens, p.pieces);
  p.runs = (tokens + p.run - 1) / p.run;
  const int64_t lists = (tokens + 3) / 4 * 4;
  int32_t* ws = static_cast<int32_t*>(workspace);
  p.key[0] = reinterpret_cast<uint32_t*>(ws);
  p.key[1] = reinterpret_cast<uint32_t*>(ws + lists);
  p.pos[0] = ws + 2 * lists;
  p.pos[1] = ws + 3 * lists;
  p.part = reinterpret_cast<float*>(ws + 4 * lists);
  hipStream_t str = (hipStream_t)stream;
  const int64_t chunks = (tokens + nvfp4::EMBED_CHUNK - 1) / nvfp4::EMBED_CHUNK;
  p.sorted = chunks > 1;
  if (tokens > 0) {
    // blocks of ids that exist (the last chunk may be short)
    const int64_t parts = (tokens + nvfp4::EMBED_RANK - 1) / nvfp4::EMBED_RANK;
    hipLaunchKernelGGL(nvfp4::embed_rank_kernel, dim3((unsigned)parts), dim3(256), 0, str, p);
    if (chunks > 1)
      hipLaunchKernelGGL(nvfp4::embed_merge_kernel, dim3((unsigned)((tokens + nvfp4::EMBED_MERGE - 1) / nvfp4::EMBED_MERGE)),
                         dim3(1024), 0, str, p);
  }
  const int64_t sum_blocks = (p.runs * p.pieces + 3) / 4;
  const int64_t fill_blocks = add == dtable ? 0 : (vocab + nvfp4::EMBED_ROWS - 1) / nvfp4::EMBED_ROWS;
  const dim3 grid((unsigned)(sum_blocks + fill_blocks)), join((unsigned)((p.runs - 1) * p.pieces));
  if (nvfp4::embed_vec(d, dout, dtable, add)) {
    hipLaunchKernelGGL(nvfp4::embed_sum_kernel<true>, grid, dim3(256), 0, str, p, sum_blocks);
    if (p.runs > 1) hipLaunchKernelGGL(nvfp4::embed_join_kernel<true>, join, dim3(64 * nvfp4::EMBED_JOIN), 0, str, p);
  } else {
    hipLaunchKernelGGL(nvfp4::embed_sum_kernel<false>, grid, dim3(256), 0, str, p, sum_blocks);
    if (p.runs > 1) hipLaunchKernelGGL(nvfp4::embed_join_kernel<false>, join, dim3(64 * nvfp4::EMBED_JOIN), 0, str, p);
  }
  return nvfp4host::launch_status();
}
