// Pages of a cache forked, taken, freed and drawn together (include/opq_attention.h).
//
// The table is all the state: a page is free if no entry names it.  Each call goes
// through four phases,
//   clear  a byte a page,
//   mark   the pages that the new table keeps (a wave a row),
//   plan   the rows' needs added up, the free pages listed (one workgroup),
//   write  the new table,
// as four kernels, or for small tables as one workgroup with barriers between.  What is
// counted are places in a fixed order (rows, columns, page ids), so nothing depends on
// who comes first: marks are stores of one value, and the one atomic takes a minimum.
// (Bits set by atomics took 115 us for the 1024 x 300 entries of rows that share
// prompts, where bytes take 5: the atomics of different XCDs on one word meet in memory.)
#include <algorithm>

#include "attention_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kNoRow = 0x7FFFFFFF;
// One workgroup: what it keeps lies in LDS, which bounds the pages, and its sixteen waves take the rows in
// turn, which bounds those.  One workgroup / four kernels, us in a graph, 64 columns and 4096
// pages: 32 rows resized 6.2/10.1, forked 6.8/11.1; 96 rows 9.2/9.8, 11.0/11.5; 128 rows 10.9/9.9,
// 13.2/11.5; 512 rows 32/10.6, 39/12.4 (launched one by one the four take 2 to 3 more).  A
// compaction goes by entries: 4096 of them 6.5/10.3, 12288 9.7/10.4, 16384 11.2/10.4, 32768 17.4/10.6.
constexpr int kOnePages = 16384;
constexpr int64_t kOneEntries = 16384;
constexpr int kOneRows = 96;

struct Space {
  uint8_t* named;   // [words * 32] 1: pages named in full (fork), or named at all
  uint8_t* part;    // [words * 32] 1: fork: pages that rows end in, partly filled
  uint32_t* words;  // [words] the pages in use, a bit each
  int32_t* first;   // [pages] fork: the first row that ends in the page; compact: where it moves
  int32_t* free;    // [pages] free pages in order, as many as are needed
  int32_t* from;    // [rows] old row of each new one, any for an empty one
  int32_t* tokens;  // [rows] its tokens
  int32_t* row;     // [rows] resize: entries lacking, then the row's first place in `free`;
                    // fork: the page the row ends in, then its place in `free`; -1: none
  int32_t* total;   // [2] pages needed, pages free
};

// Work spread over threads: this one's index and their number.
struct Me {
  int64_t thread, threads;
  __device__ int lane() const { return threadIdx.x & (kWave - 1); }
  __device__ int64_t wave() const { return thread / kWave; }
  __device__ int64_t waves() const { return threads / kWave; }
};

__device__ __forceinline__ bool named(const PagesArgs& a, int id) { return id >= 0 && id < a.pages; }
__device__ __forceinline__ int entries_of(const PagesArgs& a, int tokens) {
  return (int)(((int64_t)tokens + a.page - 1) / a.page);
}

template <PagesCall CALL>
__device__ void clear(const PagesArgs& a, const Space& s, Me me) {
  const int words = (a.pages + 31) / 32;
  for (int64_t i = me.thread; i < 2 * words; i += me.threads) {
    reinterpret_cast<uint4*>(s.named)[i] = make_uint4(0, 0, 0, 0);
    if (CALL == PagesCall::kFork) reinterpret_cast<uint4*>(s.part)[i] = make_uint4(0, 0, 0, 0);
  }
  if (CALL == PagesCall::kFork)
    for (int64_t i = me.thread; i < a.pages; i += me.threads) s.first[i] = kNoRow;
  if (CALL != PagesCall::kCompact)  // what each row is made from, looked up once
    for (int64_t row = me.thread; row < a.new_rows; row += me.threads) {
      const int from = CALL == PagesCall::kFork ? a.parents[row] : (int)row;
      const bool some = from >= 0 && from < a.rows;
      s.from[row] = some ? from : 0;
      s.tokens[row] = some ? (int)min((int64_t)max(a.lens[from], 0), (int64_t)a.columns * a.page) : 0;
    }
}

template <PagesCall CALL>
__device__ void mark(const PagesArgs& a, const Space& s, Me me) {
  if constexpr (CALL == PagesCall::kCompact) {
    const int64_t entries = (int64_t)a.rows * a.columns;
    for (int64_t i = me.thread; i < entries; i += me.threads)
      if (named(a, a.table[i])) s.named[a.table[i]] = 1;
    return;
  }
  for (int64_t row = me.wave(); row < a.new_rows; row += me.waves()) {
    if constexpr (CALL == PagesCall::kResize) {
      const int32_t* in = a.table + row * a.columns;
      const int need = entries_of(a, s.tokens[row]);
      int lack = 0;
      for (int c0 = 0; c0 < need; c0 += kWave) {
        const int c = c0 + me.lane();
        const int id = c < need ? in[c] : 0;
        if (c < need && named(a, id)) s.named[id] = 1;
        lack += __popcll(__ballot(c < need && !named(a, id)));
      }
      if (me.lane() == 0) s.row[row] = lack;
    } else {
      const int tokens = s.tokens[row], full = tokens / a.page;
      const int32_t* in = a.table + (int64_t)s.from[row] * a.columns;
      for (int c = me.lane(); c < full; c += kWave)
        if (named(a, in[c])) s.named[in[c]] = 1;
      if (me.lane() == 0) {
        const int id = tokens % a.page ? in[full] : -1;
        s.row[row] = named(a, id) ? id : -1;
        if (named(a, id)) {
          atomicMin(s.first + id, (int)row);
          s.part[id] = 1;
        }
      }
    }
  }
}

// This thread's value added over the threads before it (exclusive), and over all.
__device__ __forceinline__ int scan(int v, int* s_sum, int* all) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int up = v;
  for (int off = 1; off < kWave; off <<= 1) {
    const int o = __shfl_up(up, off, kWave);
    if (lane >= off) up += o;
  }
  __syncthreads();  // the sums of the last scan are read
  if (lane == kWave - 1) s_sum[wave] = up;
  __syncthreads();
  int before = up - v, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / kWave; ++w) {
    if (w < wave) before += s_sum[w];
    total += s_sum[w];
  }
  *all = total;
  return before;
}

// The bits of 32 bytes that are 0 or 1.
__device__ __forceinline__ uint32_t bits_of(const uint8_t* bytes) {
  const uint4* v = reinterpret_cast<const uint4*>(bytes);
  const uint4 a = v[0], b = v[1];
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    bits |= ((x[i] & 1u) | (x[i] >> 7 & 2u) | (x[i] >> 14 & 4u) | (x[i] >> 21 & 8u)) << (4 * i);
  return bits;
}
// Of the ids of word w those below `pages`.
__device__ __forceinline__ uint32_t word_mask(int pages, int w) {
  const int left = pages - w * 32;
  return left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
}

template <PagesCall CALL>
__device__ void plan(const PagesArgs& a, const Space& s, int* s_sum) {
  const int tid = threadIdx.x;
  const int words = (a.pages + 31) / 32;
  const int per = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
  // pages that a row needs; the first rows' are on their way while the words are made
  const auto needs = [&](int64_t row) {
    if (CALL == PagesCall::kCompact || row >= a.new_rows) return 0;
    const int v = s.row[row];
    if (CALL == PagesCall::kResize) return v;
    return v >= 0 && (s.named[v] || s.first[v] != (int)row) ? 1 : 0;
  };
  const int soon = needs(tid);
  int all, mine = 0;  // words w0 .. w1 - 1 are this thread's alone
  for (int w = w0; w < w1; ++w) {
    uint32_t bits = bits_of(s.named + w * 32);
    if (CALL == PagesCall::kFork) bits |= bits_of(s.part + w * 32);
    s.words[w] = bits;
    mine += __popc(bits);
  }
  if constexpr (CALL == PagesCall::kCompact) {
    scan(mine, s_sum, &all);
    const int used = all;
    int beyond = 0, holes = 0;
    for (int w = w0; w < w1; ++w) {
      const uint32_t low = word_mask(used, w), bits = s.words[w];  // ids below `used`
      beyond += __popc(bits & ~low);
      holes += __popc(~bits & low);
    }
    int moves;
    int at = scan(beyond, s_sum, &moves);
    for (int w = w0; w < w1; ++w)
      for (uint32_t b = s.words[w] & ~word_mask(used, w); b; b &= b - 1) a.src[at++] = w * 32 + __ffs(b) - 1;
    at = scan(holes, s_sum, &all);  // as many
    for (int w = w0; w < w1; ++w)
      for (uint32_t b = ~s.words[w] & word_mask(used, w); b; b &= b - 1) a.dst[at++] = w * 32 + __ffs(b) - 1;
    __syncthreads();
    for (int i = tid; i < a.moves; i += kPlanThreads) {
      if (i < moves) s.first[a.src[i]] = a.dst[i];
      else a.src[i] = a.dst[i] = -1;
    }
    if (tid == 0) s.total[0] = *a.result = used;
    return;
  }
  int needed = 0;
  for (int64_t r0 = 0; r0 < a.new_rows; r0 += kPlanThreads) {
    const int64_t row = r0 + tid;
    const int v = r0 ? needs(row) : soon;
    const int before = scan(v, s_sum, &all);
    if (row < a.new_rows) s.row[row] = CALL == PagesCall::kFork && !v ? -1 : needed + before;
    needed += all;
  }
  const int ids = max(0, min(a.pages, w1 * 32) - w0 * 32);
  int at = scan(ids - mine, s_sum, &all);
  for (int w = w0; w < w1 && at < needed; ++w)
    for (uint32_t b = ~s.words[w] & word_mask(a.pages, w); b && at < needed; b &= b - 1)
      s.free[at++] = w * 32 + __ffs(b) - 1;
  if (tid == 0) {
    s.total[0] = needed;
    s.total[1] = all;
    *a.result = max(0, needed - all);
  }
}

template <PagesCall CALL>
__device__ void write(const PagesArgs& a, const Space& s, Me me) {
  if constexpr (CALL == PagesCall::kCompact) {
    const int used = s.total[0];
    const int64_t entries = (int64_t)a.rows * a.columns;
    for (int64_t i = me.thread; i < entries; i += me.threads) {
      const int id = a.table[i];
      a.out[i] = !named(a, id) ? -1 : id < used ? id : s.first[id];
    }
    return;
  }
  const int free = s.total[1];
  for (int64_t row = me.wave(); row < a.new_rows; row += me.waves()) {
    int32_t* out = a.out + row * a.columns;
    int at = s.row[row];
    if constexpr (CALL == PagesCall::kResize) {
      const int32_t* in = a.table + row * a.columns;
      const int need = entries_of(a, s.tokens[row]);
      for (int c0 = 0; c0 < a.columns; c0 += kWave) {
        const int c = c0 + me.lane();
        int id = c < need ? in[c] : -1;
        const bool lacks = c < need && !named(a, id);
        const uint64_t mask = __ballot(lacks);
        const int k = at + __popcll(mask & ((uint64_t(1) << me.lane()) - 1));
        if (lacks) id = k < free ? s.free[k] : -1;
        if (c < a.columns) out[c] = id;
        at += __popcll(mask);
      }
    } else {
      const int tokens = s.tokens[row], need = entries_of(a, tokens);
      const int32_t* in = a.table + (int64_t)s.from[row] * a.columns;
      const int fresh = at >= 0 && at < free ? s.free[at] : -1;
      for (int c = me.lane(); c < a.columns; c += kWave) {
        int id = c < need ? in[c] : -1;
        if (!named(a, id)) id = -1;
        if (c == need - 1 && at >= 0) id = fresh;
        out[c] = id;
      }
      if (me.lane() == 0) {
        a.src[row] = fresh >= 0 ? in[need - 1] : -1;
        a.dst[row] = fresh;
        a.out_lens[row] = tokens;
      }
    }
  }
}

__device__ __forceinline__ Me in_grid() {
  return {(int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x};
}

template <PagesCall CALL>
__global__ __launch_bounds__(kRowThreads) void pages_clear(PagesArgs a, Space s) {
  clear<CALL>(a, s, in_grid());
}
template <PagesCall CALL>
__global__ __launch_bounds__(kRowThreads) void pages_mark(PagesArgs a, Space s) {
  mark<CALL>(a, s, in_grid());
}
template <PagesCall CALL>
__global__ __launch_bounds__(kPlanThreads) void pages_plan(PagesArgs a, Space s) {
  __shared__ int s_sum[kPlanThreads / kWave];
  plan<CALL>(a, s, s_sum);
}
template <PagesCall CALL>
__global__ __launch_bounds__(kRowThreads) void pages_write(PagesArgs a, Space s) {
  write<CALL>(a, s, in_grid());
}

template <PagesCall CALL>
__global__ __launch_bounds__(kPlanThreads) void pages_one(PagesArgs a, Space s) {
  __shared__ __attribute__((aligned(16))) uint8_t s_named[kOnePages];
  __shared__ __attribute__((aligned(16))) uint8_t s_part[CALL == PagesCall::kFork ? kOnePages : 16];
  __shared__ int32_t s_first[kOnePages];
  __shared__ int32_t s_rows[CALL == PagesCall::kCompact ? 1 : 3][kOneRows];
  __shared__ int32_t s_total[2];
  __shared__ int s_sum[kPlanThreads / kWave];
  const Me me{(int64_t)threadIdx.x, kPlanThreads};
  s.named = s_named;
  s.part = s_part;
  s.first = s.free = s_first;  // the free pages are listed when nobody asks for first rows any more
  s.from = s_rows[0];
  if constexpr (CALL != PagesCall::kCompact) {
    s.tokens = s_rows[1];
    s.row = s_rows[2];
  }
  s.total = s_total;
  clear<CALL>(a, s, me);
  __syncthreads();
  mark<CALL>(a, s, me);
  __syncthreads();
  plan<CALL>(a, s, s_sum);
  __syncthreads();
  write<CALL>(a, s, me);
}

size_t up256(size_t b) { return (b + 255u) & ~size_t(255); }

template <PagesCall CALL>
hipError_t launch(const PagesArgs& a, const Space& s, hipStream_t stream) {
  const int64_t entries = (int64_t)a.new_rows * a.columns;
  if (a.pages <= kOnePages && entries <= kOneEntries && (CALL == PagesCall::kCompact || a.new_rows <= kOneRows)) {
    hipLaunchKernelGGL(pages_one<CALL>, dim3(1), dim3(kPlanThreads), 0, stream, a, s);
    return hipGetLastError();
  }
  const auto blocks = [](int64_t threads) {
    return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>((threads + kRowThreads - 1) / kRowThreads, 2048)));
  };
  const dim3 rows = blocks(CALL == PagesCall::kCompact ? entries : (int64_t)a.new_rows * kWave);
  hipLaunchKernelGGL(pages_clear<CALL>, blocks(std::max<int64_t>(a.new_rows, CALL == PagesCall::kFork ? a.pages : (a.pages + 15) / 16)),
                     dim3(kRowThreads), 0, stream, a, s);
  hipLaunchKernelGGL(pages_mark<CALL>, rows, dim3(kRowThreads), 0, stream, a, s);
  hipLaunchKernelGGL(pages_plan<CALL>, dim3(1), dim3(kPlanThreads), 0, stream, a, s);
  hipLaunchKernelGGL(pages_write<CALL>, rows, dim3(kRowThreads), 0, stream, a, s);
  return hipGetLastError();
}

}  // namespace

size_t pages_workspace_bytes(int64_t rows, int64_t pages) {
  const size_t words = (size_t)(pages + 31) / 32, ids = (size_t)pages * 4;
  return 2 * up256(words * 32) + up256(words * 4) + 2 * up256(ids) + 3 * up256((size_t)rows * 4) + 256;
}

hipError_t launch_pages(PagesCall call, const PagesArgs& a, hipStream_t stream) {
  const size_t words = (size_t)(a.pages + 31) / 32;
  char* w = a.workspace;
  auto take = [&](size_t bytes) {
    char* here = w;
    w += up256(bytes);
    return here;
  };
  Space s;
  s.total = reinterpret_cast<int32_t*>(take(8));
  s.named = reinterpret_cast<uint8_t*>(take(words * 32));
  s.part = reinterpret_cast<uint8_t*>(take(words * 32));
  s.words = reinterpret_cast<uint32_t*>(take(words * 4));
  s.first = reinterpret_cast<int32_t*>(take((size_t)a.pages * 4));
  s.free = reinterpret_cast<int32_t*>(take((size_t)a.pages * 4));
  s.from = reinterpret_cast<int32_t*>(take((size_t)a.new_rows * 4));
  s.tokens = reinterpret_cast<int32_t*>(take((size_t)a.new_rows * 4));
  s.row = reinterpret_cast<int32_t*>(take((size_t)a.new_rows * 4));
  switch (call) {
    case PagesCall::kResize: return launch<PagesCall::kResize>(a, s, stream);
    case PagesCall::kFork: return launch<PagesCall::kFork>(a, s, stream);
    default: return launch<PagesCall::kCompact>(a, s, stream);
  }
}

}  // namespace opq
