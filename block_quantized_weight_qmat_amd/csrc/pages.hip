// pages.hip — page tables, slots and positions of a step from the requests'
// lengths (include/qmat.h: qmat_page_step).
//
// Four prefix sums over the sequences (tokens asked for, pages given back,
// pages asked for, pages and tokens granted), then one independent number for each page
// and token. All of it is small and waits for itself: a decode step of 64
// requests reads and writes a few KB, so what counts is the length of the
// chain of loads and barriers, and the number of launches: 48 sequences 4.2 us, 200
// sequences with 60000 rows of tokens 7.6, 1000 with as many 11.9, 4000 with 4000 rows 36.
//
// A sequence that does not fit its table row asks for its tokens like any other (the caller takes it
// out), but for no pages: it will never get one.
//
// One workgroup goes through the sequences, a thread for each, since the sums need every
// sequence, and lengths, table and stack are changed in place, which no other workgroup
// may see half done. Up to 256 sequences it has 256 threads (48 sequences 4 us, with 1024
// threads 7: every barrier waits for all waves), else 1024; more sequences are taken 1024 at a
// time, twice (pages given back have to be known before one is granted).
// The tokens' rows: a few for each of its threads (48 sequences, 600 rows: 5.5 us, 6.2 in a
// second kernel), else by a second kernel with as many workgroups as they need (2048 rows:
// 6.7 us, 8.9 in the first).
//
// Where a granted page comes from follows from the prefix sum alone: the k-th
// one in the order of (sequence, page) is stack entry top - 1 - k. So a token
// finds its page in the table (pages held before) or in the stack, and none
// waits for a page that another thread writes.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

// What a token's row needs of its sequence (in LDS, or 16 bytes each of the
// workspace).
struct Seq {
  int32_t kept;   // cells kept
  int32_t old;    // pages held before
  int32_t first;  // pages granted to the sequences before this one
  int32_t unused;
};

// What it needs of the step (in front of the workspace).
struct Step {
  int64_t tokens, top;
};

// Inclusive prefix sums of kN numbers over the workgroup's threads, in place;
// total: of all of them. s: kN * kThreads / 64 numbers of LDS.
template <int kThreads, int kN>
__device__ __forceinline__ void block_scan(int64_t (&v)[kN], int64_t (&total)[kN], int64_t* s) {
  constexpr int kWaves = kThreads / kWave;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t o = __shfl_up(v[i], d, kWave);
      if (lane >= d) v[i] += o;
    }
  }
  __syncthreads();  // what was in s before is read no more
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (lane == 63) s[i * kWaves + wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    total[i] = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) v[i] += total[i];
      total[i] += s[i * kWaves + w];
    }
  }
}

struct Lengths {
  int64_t kept, goal;
  int32_t old, now;  // pages
  bool fits;         // its row of the table
};

__device__ __forceinline__ Lengths lengths(const qmat_page_args& a, int64_t b, int shift) {
  Lengths l;
  const int64_t most = a.pages_per_seq << shift;
  int64_t held = a.kv_len[b];
  held = held < 0 ? 0 : held > most ? most : held;
  const int64_t keep = a.keep == nullptr ? held : a.keep[b];
  l.kept = keep < 0 ? 0 : keep < held ? keep : held;
  const int64_t add = a.add[b];
  l.goal = l.kept + (add < 0 ? 0 : add);
  const int64_t up = (1LL << shift) - 1;
  l.fits = l.goal <= most;
  l.old = (int32_t)((held + up) >> shift);
  l.now = l.fits ? (int32_t)((l.goal + up) >> shift) : l.old;
  return l;
}

// First index in v[0 .. n) with v[index] > x; v does not decrease.
template <typename V>
__device__ __forceinline__ int upper(const V* v, int n, V x) {
  int lo = 0;
  while (n > 0) {
    const int half = n >> 1;
    if (v[lo + half] <= x) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return lo;
}

// Row t: slot, position and sequence of token t, and the table's entry where the
// token is the first on a granted page (a granted page lies behind all cells
// kept, so its first cell is a new token). ends[b]: tokens up to sequence b's last.
__device__ __forceinline__ void token_row(const qmat_page_args& a, const int32_t* ends,
                                          const Seq* seqs, const Step& step, int shift, int64_t t) {
  int32_t slot = -1, pos = 0, seq = -1;
  if (t < step.tokens) {
    const int b = upper(ends, (int)a.n_seqs, (int32_t)t);
    const Seq s = seqs[b];
    seq = b;
    pos = s.kept + (int32_t)t - (b > 0 ? ends[b - 1] : 0);
    const int32_t j = pos >> shift, cell = pos & ((1 << shift) - 1);
    int32_t page;
    if (j < s.old) {
      page = a.page_table[b * a.pages_per_seq + j];
    } else {
      page = a.free_pages[step.top - 1 - (s.first + j - s.old)];
      if (cell == 0) a.page_table[b * a.pages_per_seq + j] = page;
    }
    if (page >= 0 && page < a.pages) slot = (page << shift) + cell;
  }
  a.slots[t] = slot;
  if (a.positions != nullptr) a.positions[t] = pos;
  if (a.token_seq != nullptr) a.token_seq[t] = seq;
}

// kOne: at most kThreads sequences. Without a step_out this kernel writes the tokens'
// rows (kOne only).
template <int kThreads, bool kOne>
__global__ __launch_bounds__(kThreads) void page_step_kernel(qmat_page_args a, int shift,
                                                             Step* step_out, Seq* seqs_out) {
  __shared__ int64_t sums[2 * kThreads / kWave];
  __shared__ int64_t back_ends[kThreads];  // pages given back up to a sequence's last
  __shared__ int32_t back_from[kThreads];  // its first page given back
  __shared__ int32_t ends[kOne ? kThreads : 1];
  __shared__ Seq seqs[kOne ? kThreads : 1];
  const int tid = threadIdx.x;
  const int64_t free = a.free_count[0];
  const int64_t count = free < 0 ? 0 : free > a.pages ? a.pages : free;

  // Tokens asked for (prefix sums), whether that fits, and the pages given
  // back and asked for. before: tokens asked for by the chunks before.
  struct Asked {
    Lengths l;
    int64_t add, back, need;
    bool in, fits;
  };
  const auto ask = [&](int64_t b, int64_t& before) {
    Asked q = {};
    q.in = b < a.n_seqs;
    if (q.in) q.l = lengths(a, b, shift);
    q.add = q.l.goal - q.l.kept;
    int64_t v[1] = {q.add}, total[1];
    block_scan<kThreads>(v, total, sums);
    q.fits = q.in && q.l.fits && (q.add == 0 || before + v[0] <= a.max_tokens);
    before += total[0];
    q.back = q.fits && q.l.old > q.l.now ? q.l.old - q.l.now : 0;
    q.need = q.fits && q.l.now > q.l.old ? q.l.now - q.l.old : 0;
    return q;
  };

  int64_t back = 0;
  if constexpr (!kOne) {
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
      int64_t v[1] = {ask(b0 + tid, before).back}, total[1];
      block_scan<kThreads>(v, total, sums);
      back += total[0];
    }
  }
  int64_t asked_tokens = 0, asked_pages = 0, back_before = 0, top = count, tokens = 0, pages = 0;
  for (int64_t b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
    const int64_t b = b0 + tid;
    const Asked q = ask(b, asked_tokens);
    int64_t v[2] = {q.back, q.need}, total[2];
    block_scan<kThreads>(v, total, sums);
    if constexpr (kOne) back = total[0];
    top = count + back < a.pages ? count + back : a.pages;
    back_ends[tid] = v[0];
    back_from[tid] = q.l.now;
    const int64_t chunk_back = total[0];
    // whoever asks for pages after one that did not get them does not either,
    // so the pages granted before are the pages asked for before
    const int64_t first = asked_pages + v[1] - q.need;
    const bool ok = q.fits && (q.need == 0 || first + q.need <= top);
    asked_pages += total[1];
    v[0] = ok ? q.add : 0;
    v[1] = ok ? q.need : 0;
    block_scan<kThreads>(v, total, sums);
    const int32_t end = (int32_t)(tokens + v[0]);
    tokens += total[0];
    pages += total[1];
    // the pages given back, the first one highest
    for (int64_t r = tid; r < chunk_back; r += kThreads) {
      const int k = upper(back_ends, kThreads, r);
      const int64_t j = back_from[k] + (r - (k > 0 ? back_ends[k - 1] : 0));
      const int64_t at = count + back - 1 - (back_before + r);
      if (at < a.pages) a.free_pages[at] = a.page_table[(b0 + k) * a.pages_per_seq + j];
    }
    back_before += chunk_back;
    if (q.in) {
      a.status[b] = ok ? 0 : q.fits ? 2 : 1;
      a.q_start[b + 1] = end;
      if (ok) a.kv_len[b] = (int32_t)q.l.goal;
      const Seq s{(int32_t)q.l.kept, q.l.old, (int32_t)first, 0};
      if constexpr (kOne) {
        ends[tid] = end;
        seqs[tid] = s;
      }
      if (!kOne || seqs_out != nullptr) seqs_out[b] = s;
    }
  }
  const Step step{tokens, top};
  if (tid == 0) {
    a.q_start[0] = 0;
    a.free_count[0] = (int32_t)(top - pages);
    if (!kOne || step_out != nullptr) *step_out = step;
  }
  if (kOne && step_out == nullptr) {
    __syncthreads();  // ends, seqs and the pages given back
    for (int64_t t = tid; t < a.max_tokens; t += kThreads) token_row(a, ends, seqs, step, shift, t);
  }
}

constexpr int kRowThreads = 256;

__global__ __launch_bounds__(kRowThreads) void page_rows_kernel(qmat_page_args a, int shift,
                                                                const Step* step, const Seq* seqs) {
  const int64_t t = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (t < a.max_tokens) token_row(a, a.q_start + 1, seqs, *step, shift, t);
}

constexpr int kManyThreads = 1024;
constexpr int kFewThreads = 256;
constexpr int kEach = 4;  // tokens' rows of a thread, where one kernel does it all

int64_t threads(const qmat_page_args& a) { return a.n_seqs <= kFewThreads ? kFewThreads : kManyThreads; }

// A thread for each sequence and kEach rows for each thread.
bool alone(const qmat_page_args& a) { return a.n_seqs <= kManyThreads && a.max_tokens <= kEach * threads(a); }

template <int kThreads, bool kOne>
void launch(const qmat_page_args& a, int shift, Step* step, Seq* seqs, hipStream_t stream) {
  hipLaunchKernelGGL((page_step_kernel<kThreads, kOne>), dim3(1), dim3(kThreads), 0, stream, a, shift, step, seqs);
}

}  // namespace

int64_t page_workspace_bytes(const qmat_page_args& a) {
  return alone(a) ? 0 : (int64_t)sizeof(Step) + a.n_seqs * (int64_t)sizeof(Seq);
}

hipError_t launch_page_step(const qmat_page_args& a, void* workspace, hipStream_t stream) {
  int shift = 0;
  while ((1LL << shift) < a.page_size) ++shift;
  const bool all = alone(a);
  Step* step = all ? nullptr : static_cast<Step*>(workspace);
  Seq* seqs = all ? nullptr : reinterpret_cast<Seq*>(step + 1);
  a.n_seqs <= kFewThreads    ? launch<kFewThreads, true>(a, shift, step, seqs, stream)
  : a.n_seqs <= kManyThreads ? launch<kManyThreads, true>(a, shift, step, seqs, stream)
                             : launch<kManyThreads, false>(a, shift, step, seqs, stream);
  const int64_t wgs = (a.max_tokens + kRowThreads - 1) / kRowThreads;
  if (!all && wgs > 0)
    hipLaunchKernelGGL(page_rows_kernel, dim3((unsigned)wgs), dim3(kRowThreads), 0, stream, a,
                       shift, step, seqs);
  return hipGetLastError();
}

}  // namespace qmat
