// Differential attention of a ragged batch over the k8v4 cache on the 5th-generation
// tensor cores:
//
//   O_m = softmax(scale q_m K_m^T) V,  m = 1, 2,   x = O_1 - lambda O_2
//
// Both maps of a row weigh the same values, but their sums are known only when the last
// cell is scored, so each map keeps an O of its own: 2 x 256 fp32 columns a row, all of
// tensor memory.  A unit of work is therefore ONE map of a tile of 32 tokens (x the 8 query
// heads of a KV head = 256 rows) over a range of the cells: a CTA pair (tcgen05
// cta_group::2, M = 256, 128 rows per SM) keeps its O in tensor memory and sweeps the range
// in tiles of 128 cells
//   S  = Q_m K_m^T        128 lanes, N = 128 (fp32 queries in two fp16 terms: twice)
//   P  = 2^(s - ref) 2^2  online softmax in the log2 domain, fp16
//   O += P V              N = 256, V = RN((n - 8) d) in fp16
// and writes its partial rows (o, m, l); the combine joins ranges and maps.  The two maps'
// units read and convert the same V; a pair that kept both maps of 16 tokens instead would
// need both key halves too, and twice the conversions per product.
//
// Each CTA of the pair dequantises half of every tile (64 of the 128 cells of K, 128 of the
// 256 dims of V); the pair reads both halves as one operand.  P and V are rounded to fp16
// once (2^-11 of each term at most; the result is bf16; 32 cells with a block that fp16 does not hold eight
// times over count with V / 8 and 8 P, as a tile in k8v4_diff.cu), so a tile takes 8 products of 64 clocks for
// S and 8 of 128 for O where the exact kernels' two terms each would take three times the
// latter.
//
// Roles, handing over through mbarriers:
//      warps 0-7    rows: a thread per row; warps 0-3 take the even tiles, 4-7 the odd ones, so
//                   that one group's exponentials run beside the other's maxima and waits
//      warps 8-15   conversion: raw tile -> registers -> operand tiles, K (8-11) and V (12-15)
//      warp 16      (leader CTA) issues every product of the pair
//      warps 17-19  copy the raw tiles (TMA, boxes of 64, 32 or 16 cells as the page size allows; a
//                   copy takes its warp about 100 clocks to issue, and 16-cell boxes need 28 a tile)
// The issuing warp hands over whichever product is ready, S or O (in a fixed order of the two
// one waits for the other's reader: 4,096 tokens on 32,768 cells 2.53 ms against 2.03 then, without
// any rescaling): a row's thread takes its 128 scores into registers at once and frees S, and P
// has two buffers of its own.
// The reference maximum of a row moves only when a tile exceeds it by 2^10, and then its O
// is rescaled in tensor memory, which holds the pair up for about 1,100 clocks; the two groups
// hand the reference on from tile to tile.  P is kept 2^5 above it: what is less than 2^-19 of the
// reference is subnormal, and off by 2^-30 of it at most.  (That case, and with queries 10 times as large:
// 2.30 and 3.87 ms; at 2^13 and 2^2, where terms of 2^-27 are dropped, 2.26 and 3.65, at 2^8 and 2^7 2.36 and 4.04.)
// Every kChain tiles O is added to a running sum in global memory (the unit's own partial
// rows serve as its place), because the tensor core's accumulation is not rounded to
// nearest: measured 2.9e-5 after 2,048 cells in three products each, so about 4e-5 after
// kChain tiles here.
//
// The units come from a schedule that one CTA works out on the device from the lengths:
// token tiles, heaviest first within a sequence, cut into ranges so that the pairs of the
// device are evenly loaded.  Sequences of few tokens would leave most of a tile's 256 rows empty;
// where it is estimated to be faster their tokens go through the single queries' kernel
// (k8v4_diff.cu) one by one.
//
// What bounds it: the products (1,536 of a tile's about 2,700 clocks) and what the row warps do
// between them; 4,096 tokens on 32,768 cells 2.30 ms, 1.34 PFLOP/s (2.10 without the look at the blocks' sizes, the
// fence and the small weights' bits).  Short units pay 10 us each
// beside their tiles: 12 prompts of 900 tokens 229 us.
//
// Tensor memory (512 columns): S [0,128), P [128,192) and [192,256), O [256,512).
//
// Every mbarrier wait is bounded: on timeout the warp raises the CTA's failure word and
// leaves its loop; the kernel records an error, waits for its own products (bounded), frees
// its tensor memory and returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "k8v4_diff.cuh"
#include "k8v4_tc.cuh"
#include "k8v4_tma.cuh"

namespace k8v4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 128;                    // query rows per CTA (256 per pair)
constexpr int kTileN = 128;                   // cells per tile
constexpr int kRowWarps = 8;
constexpr int kConvWarp0 = kRowWarps, kVConvWarp0 = kConvWarp0 + 4, kIssueWarp = kConvWarp0 + 8, kLoadWarp0 = kIssueWarp + 1;
constexpr int kLoadWarps = 3, kThreads = 32 * (kLoadWarp0 + kLoadWarps);
// the register split waits for whole warpgroups: roles begin at multiples of four warps
static_assert(kConvWarp0 % 4 == 0 && kIssueWarp % 4 == 0 && kThreads == 32 * (kIssueWarp + 4), "roles");
constexpr int kChain = 64;                    // tiles accumulated in tensor memory (8,192 cells)
constexpr float kSlack = 10.0f, kLift = 5.0f; // log2 headroom of P above its row's reference maximum, and what P is lifted by
static_assert(kSlack + kLift <= 15.0f, "P in fp16");
constexpr uint32_t kWaitDefaultNs = 1000000000u;
// registers per thread after the split (8 row, 8 conversion and 4 other warps), out of those of
// the 20 warps that the block launches with
constexpr int kLaunchRegs = 96, kRowRegs = 160, kConvRegs = 64, kIssueRegs = 24;
static_assert(2 * kRowRegs + 2 * kConvRegs + kIssueRegs <= 5 * kLaunchRegs, "register split");

// shared memory (bytes); operand tiles 1024-byte aligned, the same in both CTAs
constexpr int kQOff = 0;                              // Q fp16 [2 chunks][128 rows][128 B]
constexpr int kKOff = kQOff + 32768;                  // K fp16, 2 buffers x [2 chunks][64 cells][128 B]
constexpr int kKBuf = 16384;
constexpr int kVOff = kKOff + 2 * kKBuf;              // V fp16, 2 buffers x [2 atoms][128 cells][128 B]
constexpr int kVBuf = 32768, kVAtom = 16384;
// K scales, kKsRing tiles x [128] f32, and as many words of odd cells.  A row frees S before it reads these, so
// the conversion of tile i, which waits for S(i - 2) and with it for S(i - 3) and S(i - 4) to be read, knows that the
// groups are in their tiles i - 3 and i - 4 and done with those up to i - 5 and i - 6: six places do.
// Four (with three raw tiles in flight, nothing else holds the conversion back) would not
constexpr int kKsRing = 8;
constexpr int kKsOff = kVOff + 2 * kVBuf;
constexpr int kRedOff = kKsOff + kKsRing * 512;             // [128] f32 each: score factors, references, sums of the two groups
constexpr int kBarOff = kRedOff + 4 * 512;
constexpr int kCtlOff = kBarOff + 256;                // tmem slot, failure word, odd cells of the ring's tiles, valid groups of the stages
constexpr int kRawOff = (kCtlOff + 64 + 1023) / 1024 * 1024;
constexpr int kSmemMax = 227 * 1024;
// a raw tile: K codes of the CTA's 64 cells (4 boxes of 16 cells x 128 B), V nibbles of the 128 cells (8 boxes),
// and the runs of K and V scales of all heads (8 groups x 128 H and 256 H bytes)
constexpr int kRawV = 8192, kRawKs = 24576;
constexpr int raw_bytes(int H) { return (kRawKs + 3 * 1024 * H + 1023) / 1024 * 1024; }
// fp32 queries: the second terms, laid out as the first, stand behind the raw tiles
constexpr int kQBytes = 32768;
constexpr int raw_stages(int H, bool q_f32) {
  const int fit = (kSmemMax - kRawOff - (q_f32 ? kQBytes : 0)) / raw_bytes(H);
  return fit < 3 ? fit : 3;
}
static_assert(kKsRing >= 6 && kKsRing <= 8 && raw_stages(2, false) == 3 && raw_stages(7, false) >= 2 && raw_stages(8, false) >= 1, "raw stages");
static_assert(raw_stages(2, true) >= 2 && raw_stages(8, true) >= 1, "raw stages");
// the epilogue reuses the operand tiles as a fp32 [128][256] row buffer
static_assert(kKsOff - kQOff >= kRows * 256 * 4, "row buffer");

// mbarriers, at kBarOff + 8 * index
enum { kBarKFull = 0, kBarVFull = 2, kBarPFull = 4, kBarSFull = 6, kBarODone = 8, kBarKsFull = 10, kBarSFree = 14,
       kBarDrain = 15, kBarRawFull = 16, kBarRawEmpty = 20, kBarRef = 24 };

constexpr uint32_t kTmemCols = 512, kPCol = 128, kPBuf = 64, kOCol = 256;

// ---------------------------------------------------------------- the schedule
constexpr int kTileTok = 32;                  // tokens of a token tile
// ranges: room for so many units more than token tiles, per pair of the device: four where there are
// few tiles, two where the tiles alone are several rounds (every unit without work costs a launch of
// two empty CTAs: 12 prompts of 900 tokens 208 us with four, 197 with two; 300 tokens behind 100,000 649 and 721),
// one where few tokens a sequence leave the tiles without work most often (8 sequences of up to
// 5 tokens 53.0 us with four, 51.4 with one)
constexpr int kMostWaves = 4, kFewWaves = 2;
struct TokenTile {
  int seq, tok0, n, splits, first, cell_tiles, vis0, most;   // vis0: cells that its first token sees (causal), or the steps' bound
};
// what a CTA pair needs to know, in one read: its tokens, its cell tiles [tile0, tile0 + n_tiles), the cells that any of its
// rows sees, and which map (bit 0) of which KV head
struct Unit {
  int seq, tok0, n, vis0, tile0, n_tiles, limit, what;
};

struct Schedule {                             // places in the workspace
  int32_t* head;                              // [0] units, [1] single queries
  float* lambdas;                             // [8 H]
  int32_t* tile_end;                          // [n_seqs] token tiles up to each sequence
  TokenTile* tiles;
  int32_t* tok_tile;                          // [n_tok], -1: no sequence's, -2 - query: a single query
  int32_t* row_seq;                           // of each single query
  int32_t* row_tok;
  int32_t* row_vis;
  DiffPieces pieces;
  Unit* units;
  float* rows;                                // partial blocks of 256 rows
};
constexpr int kMostFew = 8;                   // tokens of a sequence that may go one by one
int64_t most_rows(int n_seqs, int n_tok) { return std::min<int64_t>(n_tok, static_cast<int64_t>(kMostFew) * n_seqs); }
int64_t most_tiles(int n_seqs, int n_tok) { return n_tok / kTileTok + std::min(n_seqs, n_tok); }
int64_t more_units(int64_t base, int pairs, int n_seqs, int n_tok) {
  if (n_tok <= static_cast<int64_t>(kMostFew) * n_seqs) return pairs;
  return std::max(static_cast<int64_t>(kFewWaves) * pairs, static_cast<int64_t>(kMostWaves) * pairs - base);
}
int64_t most_units(int n_seqs, int n_tok, int max_seq_len, int H, int pairs) {
  const int64_t base = most_tiles(n_seqs, n_tok) * 2 * H;
  return std::min(base * std::max(1, (max_seq_len + kTileN - 1) / kTileN), base + more_units(base, pairs, n_seqs, n_tok));
}
// what a workspace has room for: the most that any batch within these sizes can have, so that one which was made for
// the largest batch serves all (sequences of few tokens take fewer ranges than as many tokens of one)
int64_t room_for(int n_seqs, int n_tok, int max_seq_len, int H, int pairs) {
  const int64_t base = most_tiles(n_seqs, n_tok) * 2 * H;
  return std::min(base * std::max(1, (max_seq_len + kTileN - 1) / kTileN),
                  std::max(base + static_cast<int64_t>(kFewWaves) * pairs, static_cast<int64_t>(kMostWaves) * pairs));
}
size_t place(Schedule* s, uint8_t* ws, int n_seqs, int n_tok, int max_seq_len, int H, int pairs, int num_sms) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t tiles = most_tiles(n_seqs, n_tok), units = room_for(n_seqs, n_tok, max_seq_len, H, pairs);
  Schedule t;
  t.head = reinterpret_cast<int32_t*>(take(8));
  t.lambdas = reinterpret_cast<float*>(take(sizeof(float) * kGqa * H));
  t.tile_end = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(n_seqs)));
  t.tiles = reinterpret_cast<TokenTile*>(take(sizeof(TokenTile) * tiles));
  t.tok_tile = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(n_tok)));
  const int64_t rows = most_rows(n_seqs, n_tok);
  t.row_seq = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  t.row_tok = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  t.row_vis = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(rows)));
  place_pieces(&t.pieces, take(place_pieces(nullptr, nullptr, rows * H, num_sms)), rows * H, num_sms);
  t.units = reinterpret_cast<Unit*>(take(sizeof(Unit) * units));
  t.rows = reinterpret_cast<float*>(take(static_cast<size_t>(units) * 2 * kRows * kDiffRow * sizeof(float)));
  if (s) *s = t;
  return at;
}

struct ScheduleParams {
  Schedule s;
  k8v4_diff d;
  const int32_t* offsets;
  const int32_t* lens;
  const int32_t* steps;
  int n_seqs, n_tok, max_seq_len, H, pairs;
  int64_t most, more, most_rows;                    // units, units beyond one a tile, and single queries that there is room for
  int* status;
};

__device__ __forceinline__ int scan_block(int v, int* red, int* total) {   // 1,024 threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) red[warp] = s;
  __syncthreads();
  int w = red[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(kFull, w, 31);
  const int ahead = __shfl_sync(kFull, w, max(warp - 1, 0));
  return s - v + (warp ? ahead : 0);
}

// One CTA.  Token tiles of each sequence, the last first (it sees the most cells); the range
// length that keeps the pairs of the device evenly loaded; the units.  What is searched and
// counted stays in shared memory while the lists are short (a search of a list in global
// memory is a chain of reads of 300 ns each).
constexpr int kShortList = 4096, kBuckets = 256;
__global__ void __launch_bounds__(1024, 1) diff_schedule_kernel(const ScheduleParams p) {
  __shared__ int red[32];
  __shared__ float cost_s[32];
  __shared__ int cand_s[32];
  __shared__ int top_s, few_n;
  __shared__ unsigned long long claimed_s, cells_sum_s;        // token tiles and their cell tiles: offsets that name tokens again and again pass 32 bits
  __shared__ int ends_s[kShortList], cells_s[kShortList];
  __shared__ unsigned long long few_s[kMostFew + 1];           // sixteens of cells of the sequences of so many tokens; [0] of the others' token tiles
  __shared__ int bucket_s[kBuckets];
  __shared__ uint8_t bucket_of[kShortList];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x <= kMostFew) few_s[threadIdx.x] = 0;
  if (threadIdx.x < kBuckets) bucket_s[threadIdx.x] = 0;
  if (threadIdx.x == 0) claimed_s = cells_sum_s = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Schedule& s = p.s;
  for (int t = tid; t < p.n_tok; t += 1024) s.tok_tile[t] = -1;
  // ---- lambda of each head, for the joining (a warp there that works it out for its row: 5 of 12 900-token prompts' 195 us)
  for (int hq = warp; hq < kGqa * p.H; hq += 32) {
    float l = 0.0f;
#pragma unroll 1
    for (int term = 0; term < 2; ++term) l = diff_lambda_term(p.d, hq, term, lane) - l;     // -(first - second)
    if (lane == 0) s.lambdas[hq] = p.d.lambda_init - l;
  }
  __syncthreads();
  // ---- the sequences' tokens and cells
  int* const ends = p.n_seqs <= kShortList ? ends_s : s.tile_end;
  const int per = (p.n_seqs + 1023) / 1024;
  const int b0 = min(p.n_seqs, tid * per), b1 = min(p.n_seqs, b0 + per);
  auto tokens_of = [&](int b, int& first) {
    first = p.offsets[b];
    const int end = p.offsets[b + 1];
    return first < 0 || end < first || end > p.n_tok ? -1 : end - first;
  };
  auto len_of = [&](int b) { return min(max(p.lens[b], 0), p.max_seq_len); };
  for (int b = b0; b < b1; ++b) {
    int first;
    const int n = tokens_of(b, first), len = p.lens[b];
    if (n < 0 || len < 0 || len > p.max_seq_len) record_status(p.status, K8V4_ERANGE);
    const unsigned long long t16 = (len_of(b) + 15) >> 4;
    if (n > 0) atomicAdd(few_s + (n <= kMostFew ? n : 0), n <= kMostFew ? t16 : t16 * ((n + kTileTok - 1) / kTileTok));
  }
  __syncthreads();
  // ---- up to how many tokens a sequence's go one by one: what leaves the shorter time, by rates
  // measured at 2 KV heads (16 cells of one KV head: 1.4 ns a query, 6 ns a token tile that is mostly empty; a kernel
  // that has work: 8 us and 14).  32 sequences of 8,192 cells: 81 us one by one against 228 for one token each, 221
  // against 226 for four, 313 against 229 for six.  (One warp: the conversions of 64-bit sums are slow.)
  if (warp == 0) {
    const float t = lane <= kMostFew ? static_cast<float>(few_s[lane]) : 0.f;
    float one = 0.f, tile = 0.f;
#pragma unroll 1
    for (int n = 0; n <= kMostFew; ++n) {
      const float tn = __shfl_sync(kFull, t, n);
      if (n >= 1 && n <= lane) one += 1.4f * n * tn;
      else tile += 6.f * tn;
    }
    const float cost = lane > kMostFew ? INFINITY : (one + tile) * p.H + (one > 0.f ? 8000.f : 0.f) + (tile > 0.f ? 14000.f : 0.f);
    float best = cost;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) best = fminf(best, __shfl_xor_sync(kFull, best, o));
    if (lane == 0) top_s = 0;
    const int at_best = 31 - __clz(__ballot_sync(kFull, cost == best));
    if (lane == 0) few_n = at_best;
  }
  __syncthreads();
  const int few = few_n;
  // ---- their queries, and the others' token tiles
  int sum = 0, rows = 0, n_tiles, n_rows;
  for (int b = b0; b < b1; ++b) {
    int first;
    const int n = tokens_of(b, first);
    if (n > few) sum += (n + kTileTok - 1) / kTileTok;
    else rows += max(n, 0);
    ends[b] = sum;                                             // of this thread's sequences so far
  }
  {
    const int of_warp = __reduce_add_sync(kFull, sum);           // below 32 * 64 sequences * 2^19 tiles
    if (lane == 0 && of_warp) atomicAdd(&claimed_s, static_cast<unsigned long long>(of_warp));
  }
  const int at = scan_block(sum, red, &n_tiles);
  int row = scan_block(rows, red, &n_rows);
  for (int b = b0; b < b1; ++b) {
    ends[b] += at;
    int first;
    const int n = tokens_of(b, first);
    if (n > few) continue;
    const int len = len_of(b);
    for (int k = 0; k < n; ++k, ++row) {
      if (row >= p.most_rows) break;
      int vis = p.steps ? p.steps[first + k] : max(len - n + k + 1, 0);
      if (vis < 0 || vis > len) {
        record_status(p.status, K8V4_ERANGE);
        vis = vis < 0 ? 0 : len;
      }
      s.row_seq[row] = b;
      s.row_tok[row] = first + k;
      s.row_vis[row] = vis;
      s.tok_tile[first + k] = -2 - row;
    }
  }
  // offsets that do not follow one another can claim more tiles than there is room for
  if (claimed_s > static_cast<unsigned long long>(p.n_tok / kTileTok + min(p.n_seqs, p.n_tok))) {
    if (tid == 0) record_status(p.status, K8V4_ERANGE);
    n_tiles = 0;
  }
  if (n_tiles == 0) {
    if (tid == 0) {
      s.head[0] = 0;
      s.head[1] = static_cast<int>(min(static_cast<int64_t>(n_rows), p.most_rows));
    }
    return;
  }
  __syncthreads();
  // ---- each tile's tokens and cells
  const bool brief = n_tiles <= kShortList;
  unsigned long long cells = 0;
  int top = 0;
  for (int i = tid; i < n_tiles; i += 1024) {
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > i) hi = mid;
      else lo = mid + 1;
    }
    TokenTile t;
    t.seq = lo;
    int first;
    const int n = tokens_of(lo, first);
    const int j = ends[lo] - 1 - i;                            // the last tile first
    t.tok0 = first + j * kTileTok;
    t.n = min(kTileTok, n - j * kTileTok);
    int len = p.lens[lo];
    if (len < 0 || len > p.max_seq_len) {
      len = len < 0 ? 0 : p.max_seq_len;                       // (recorded above)
    }
    t.vis0 = len - n + j * kTileTok + 1;
    int most = max(t.vis0 + t.n - 1, 0);
    if (p.steps) {
      most = 0;
      for (int k = 0; k < t.n; ++k) {
        const int v = p.steps[t.tok0 + k];
        if (v < 0 || v > len) record_status(p.status, K8V4_ERANGE);
        most = max(most, min(v, len));
      }
      t.vis0 = len;
    }
    t.cell_tiles = (most + kTileN - 1) / kTileN;
    t.splits = t.first = 0;
    t.most = most;
    s.tiles[i] = t;
    if (brief) cells_s[i] = t.cell_tiles;
    for (int k = 0; k < t.n; ++k) s.tok_tile[t.tok0 + k] = i;
    cells += t.cell_tiles;
    top = max(top, t.cell_tiles);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) cells += __shfl_xor_sync(kFull, cells, o);
  if (lane == 0 && cells) atomicAdd(&cells_sum_s, cells);        // (an atomic for each thread with a tile: 360 in line, 4 us)
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) atomicMax(&top_s, top);
  __syncthreads();
  const float total = static_cast<float>(cells_sum_s);
  top = max(top_s, 1);
  // ---- the range length: 32 candidates from what makes all the units that there is room for to no
  // cut at all, each worked out by a warp: rounds x (range + a unit's fixed cost)
  const float units_per = 2.0f * p.H;
  const int least = max(1, min(top, static_cast<int>(ceilf(units_per * total / static_cast<float>(p.more)))));
  // (what a unit takes beside its tiles: launch, query, first products 4.7 us, O and its rows 4.3, hand-over 1, at
  // 1.29 us a tile: 12 prompts of 900 tokens)
  constexpr float kFixedTiles = 8.0f;
  int range = top;
  if (brief) {                                                 // long lists are not cut
    const int cand = max(least, min(top, static_cast<int>(ceilf(least * exp2f(log2f(static_cast<float>(top) / least) * warp / 31.0f)))));
    int units = 0;
    for (int i = lane; i < n_tiles; i += 32) units += (cells_s[i] + cand - 1) / cand;
    units = __reduce_add_sync(kFull, units);
    if (lane == 0) cand_s[warp] = cand, cost_s[warp] = ceilf(units * units_per / p.pairs) * (cand + kFixedTiles);
    __syncthreads();
    float best = cost_s[lane];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) best = fminf(best, __shfl_xor_sync(kFull, best, o));
    range = cand_s[31 - __clz(__ballot_sync(kFull, cost_s[lane] == best))];
  }
  // ---- the units, the longest first, so that the pairs finish together (40 sequences of up to 300 tokens: 154 us in the
  // tiles' order, 144 so); a long list stays in the tiles' order
  int all;
  if (brief) {
    int* const splits_s = ends_s;                              // (the sequences' ends are done with)
    for (int i = tid; i < n_tiles; i += 1024) {
      const int sp = splits_s[i] = (cells_s[i] + range - 1) / range;
      if (sp == 0) continue;
      const int len = (cells_s[i] + sp - 1) / sp;              // the tiles of a unit, at most `range`
      const int b = kBuckets - 1 - static_cast<int>(static_cast<float>(len) * (kBuckets - 1) / range);
      bucket_of[i] = static_cast<uint8_t>(max(b, 0));
      atomicAdd(bucket_s + bucket_of[i], sp * 2 * p.H);
    }
    __syncthreads();
    const int mine = tid < kBuckets ? bucket_s[tid] : 0;
    const int before = scan_block(mine, red, &all);
    if (tid < kBuckets) bucket_s[tid] = before;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += 1024) {                // (the order within a bucket moves where rows are kept, not what is in them)
      const int sp = splits_s[i];
      s.tiles[i].splits = sp;
      s.tiles[i].first = sp ? atomicAdd(bucket_s + bucket_of[i], sp * 2 * p.H) : 0;
    }
  } else {
    const int tiles_per = (n_tiles + 1023) / 1024;
    const int i0 = min(n_tiles, tid * tiles_per), i1 = min(n_tiles, i0 + tiles_per);
    int mine = 0;
    for (int i = i0; i < i1; ++i) mine += (s.tiles[i].cell_tiles + range - 1) / range * 2 * p.H;
    int u = scan_block(mine, red, &all);
    for (int i = i0; i < i1; ++i) {
      const int sp = (s.tiles[i].cell_tiles + range - 1) / range;
      s.tiles[i].splits = sp;
      s.tiles[i].first = u;
      u += 2 * p.H * sp;
    }
  }
  all = static_cast<int>(min(static_cast<int64_t>(all), p.most));
  __syncthreads();
  for (int i = warp; i < n_tiles; i += 32) {                   // a warp writes a tile's units
    const TokenTile t = s.tiles[i];
    if (t.splits == 0) continue;
    const int len = (t.cell_tiles + t.splits - 1) / t.splits, units = 2 * p.H * t.splits;
    for (int v = lane; v < units && t.first + v < all; v += 32) {
      const int k = v / t.splits, c = v - k * t.splits;
      s.units[t.first + v] = Unit{t.seq, t.tok0, t.n, t.vis0, c * len, min(len, t.cell_tiles - c * len), t.most, k};
    }
  }
  if (tid == 0) {
    s.head[0] = all;
    s.head[1] = static_cast<int>(min(static_cast<int64_t>(n_rows), p.most_rows));
  }
}

// ---------------------------------------------------------------- waits
// mbar_wait for waits that nearly always end soon: the barrier's own bounded sleep first, the
// clock only behind it
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, uint32_t limit_ns) {
  if (limit_ns >= 1000u && mbar_try(bar, parity, 20000u)) return true;
  return mbar_wait(bar, parity, limit_ns);
}

// ---------------------------------------------------------------- pair PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
// (no wider release than the CTA's: what the tensor core reads is made visible by the proxy and
// tcgen05 fences ahead of the arrival)
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// completion of this thread's products so far -> the barrier at this offset of both CTAs
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// a barrier over the row warps that also ORs a predicate
__device__ __forceinline__ bool rows_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void rows_barrier() { asm volatile("barrier.cta.sync 2, 256;" ::: "memory"); }
// 128 consecutive fp32 columns of this thread's TMEM lane: four loads in flight, one wait
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float v[128]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float* x = v + 32 * h;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
          "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
          "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
          "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
        : "r"(taddr + 32 * h)
        : "memory");
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) asm volatile("" : "+f"(v[i]));       // no use of them moves ahead of the wait
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t v[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float v[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]),
        "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]),
        "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// A word of nibble bytes b0..b3 -> fp16 pairs of V = RN((n - 8) d): lo {b0, b2}, {b1, b3} of the
// low nibbles, hi of the high ones.  0x640n is 1024 + n and 0x64n0 is 1024 + 16 n in fp16;
// 1024 + n - 1032 and (1024 + 16 n) / 16 - 72 are both n - 8, exactly.  (Elements 1 and
// 2 of each four come out swapped; the rows are put right as they are written.)
__device__ __forceinline__ void nib_word(uint32_t r, __half2 d2, uint32_t lo[2], uint32_t hi[2]) {
  const uint32_t r8 = r >> 8;
  const __half2 m1032 = __halves2half2(__ushort_as_half(0xe408), __ushort_as_half(0xe408));     // -1032
  const __half2 c16th = __halves2half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));     // 1/16
  const __half2 m72 = __halves2half2(__ushort_as_half(0xd480), __ushort_as_half(0xd480));       // -72
  const uint32_t t0 = (r & 0x000f000fu) | 0x64006400u, t1 = (r8 & 0x000f000fu) | 0x64006400u;
  const uint32_t t2 = (r & 0x00f000f0u) | 0x64006400u, t3 = (r8 & 0x00f000f0u) | 0x64006400u;
  const __half2 v0 = __hmul2(__hadd2(*reinterpret_cast<const __half2*>(&t0), m1032), d2);
  const __half2 v1 = __hmul2(__hadd2(*reinterpret_cast<const __half2*>(&t1), m1032), d2);
  const __half2 v2 = __hmul2(__hfma2(*reinterpret_cast<const __half2*>(&t2), c16th, m72), d2);
  const __half2 v3 = __hmul2(__hfma2(*reinterpret_cast<const __half2*>(&t3), c16th, m72), d2);
  lo[0] = *reinterpret_cast<const uint32_t*>(&v0);
  lo[1] = *reinterpret_cast<const uint32_t*>(&v1);
  hi[0] = *reinterpret_cast<const uint32_t*>(&v2);
  hi[1] = *reinterpret_cast<const uint32_t*>(&v3);
}

// ---------------------------------------------------------------- the kernel
struct PairParams {
  CacheView C;
  const void* q;            // [n_tok][HQ][256]
  int q_f32;
  const int32_t* pt;        // [n_seqs][max_pages]
  int64_t max_pages;
  const int32_t* steps;     // or null
  Schedule s;
  float sm_scale_log2;
  int* status;
  uint32_t wait_ns;
  FastDiv page_div;
  int stages, stage_bytes;  // raw tiles in flight
  int q_lo;                 // fp32 queries: where in shared memory the second terms stand
  int box_shift;            // log2 of the cells of a copy: 4, 5 or 6
};

// grid: 2 CTAs per unit
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    diff_pair_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PairParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const CacheView& C = p.C;
  const int HQ = C.H * kGqa;
  const int row = tid & (kRows - 1), group = tid >> 7;     // (row warps) tiles group, group + 2, ...
  const uint32_t bars = sb + kBarOff;
  volatile int* ctl = reinterpret_cast<volatile int*>(smem + kCtlOff);   // [0] tmem, [1] failed, [4..11] odd cells (a byte for each 32: bad groups, 4: large blocks), [12..14] valid groups
  float* fsc = reinterpret_cast<float*>(smem + kRedOff);                 // [128] score factors
  float* ref = fsc + kRows;                                              // [128] reference maxima
  float* sums = fsc + 2 * kRows;                                         // [2][128]
  float* ksbuf = reinterpret_cast<float*>(smem + kKsOff);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x >> 1;
  const int4* src = reinterpret_cast<const int4*>(p.s.units + unit);
  const int4 ua = __ldcg(src), ub = __ldcg(src + 1);                     // (read beside the count: one latency)
  if (unit >= __ldcg(p.s.head)) return;                                  // both CTAs of the pair
  const int seq = ua.x, tok0 = ua.y, vis0 = ua.w, tile0 = ub.x, n_tiles = ub.y;   // n_tiles >= 1
  const int limit = ub.z;                                                // cells that any row of the pair sees (those behind are neither looked up nor read)
  const int map = ub.w & 1, g = ub.w >> 1;
  const int tok_first = tok0 + 16 * static_cast<int>(rank);              // this CTA's tokens
  const int tok_n = max(0, min(16, ua.z - 16 * static_cast<int>(rank)));
  const int32_t* pt = p.pt + static_cast<int64_t>(seq) * p.max_pages;

  if (warp == kLoadWarp0) {
    int count = 0;
    if (lane < kBarPFull) count = 8;                       // K, V tiles: 4 conversion warps of both CTAs
    else if (lane < kBarSFull) count = 8;                  // P: a tile's 4 row warps of both CTAs
    else if (lane < kBarKsFull) count = 1;                 // S done, O done: one commit
    else if (lane < kBarSFree) count = 4;                  // K scales: the CTA's K conversion warps
    else if (lane == kBarSFree) count = 8;                 // S read: 4 row warps of both CTAs
    else if (lane == kBarDrain) count = 1;                 // everything done: one commit
    else if (lane < kBarRawEmpty) count = kLoadWarps;      // raw tile: the loaders, and the bytes of their copies
    else if (lane < kBarRef) count = 8;                    // raw tile read: the CTA's conversion warps
    else count = 1;                                        // a warp's references: [quarter of the rows][tile & 1]
    mbar_init(bars + 8 * lane, count);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane < 15) ctl[1 + lane] = 0;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
  }
  if (warp == kIssueWarp) tmem_alloc_pair(sb + kCtlOff, kTmemCols);

  // ---- the load warps' copies of tile i into a stage.  Warp 0 of the three takes the V rows, 1 the V scales, 2 the K rows of
  // this CTA's half and the K scales, a lane to a copy.  Page ids of four tiles, eight 16-cell groups each (those of the
  // copy that brings the group), are held one per lane, and those of the next four are on their way.
  const int which = warp - kLoadWarp0, per = p.box_shift - 4, copies = 8 >> per;   // 1 << per groups a copy
  int page_next = 0, page_mine = 0;
  auto lookup = [&](int i) -> int {
    const uint32_t c = static_cast<uint32_t>(tile0 + i + (lane >> 3)) * kTileN + 16 * ((lane & 7) >> per << per);
    if (i + (lane >> 3) >= n_tiles || c >= static_cast<uint32_t>(limit)) return INT32_MIN;        // behind the limit, or another range's
    const int64_t pidx = p.page_div.div(c);
    return pidx < p.max_pages ? __ldcg(pt + pidx) : -1;
  };
  auto load_tile = [&](int i, int stage) {
    const int H = C.H;
    if ((i & 3) == 0) {
      page_mine = page_next == INT32_MIN || (page_next >= 0 && page_next < C.n_pages) ? page_next : -1;
      page_next = lookup(i + 4);
    }
    const uint32_t dst = sb + kRawOff + stage * p.stage_bytes, bar = bars + 8 * (kBarRawFull + stage);
    const int my_group_page = __shfl_sync(kFull, page_mine, 8 * (i & 3) + (lane & 7));
    const unsigned good = __ballot_sync(kFull, my_group_page >= 0) & 255u;
    const unsigned bad = __ballot_sync(kFull, my_group_page == -1) & 255u;
    if (lane == 0) {
      if (which == 0) {
        if (bad) record_status(p.status, K8V4_ERANGE);
        ctl[12 + stage] = static_cast<int>(good | (bad << 8));
      }
      const uint32_t n = __popc(good), nk = __popc((good >> (4 * rank)) & 15u);
      mbar_expect_tx(bar, which == 0 ? n * 2048u : which == 1 ? n * 256u * H : n * 128u * H + nk * 2048u);
    }
    __syncwarp();
    // lanes 0-7 a run of 1 << per groups each; the K rows lanes 8-11
    const bool k_rows = which == 2 && lane >= 8;
    const int q = (k_rows ? 4 * static_cast<int>(rank) + ((lane & 3) << per) : lane << per) & 7;
    const int page = __shfl_sync(kFull, page_mine, 8 * (i & 3) + q);
    if (page >= 0 && (k_rows ? lane - 8 < (copies + 1) >> 1 : lane < copies)) {
      const int cell = (tile0 + i) * kTileN + 16 * q;
      const int slot = cell - static_cast<int>(p.page_div.div(static_cast<uint32_t>(cell))) * C.P;
      const uint8_t* pg = C.pages + static_cast<int64_t>(page) * C.page_bytes;
      if (which == 0) tma_load_4d(dst + kRawV + q * 2048, &tm_v, 0, g, slot, page, bar);
      else if (which == 1) bulk_load(dst + kRawKs + 1024 * H + q * 256 * H, pg + C.vs_off() + static_cast<int64_t>(slot) * 16 * H, 256 * H << per, bar);
      else if (k_rows) tma_load_4d(dst + (q & 3) * 2048, &tm_k, 128 * map, g, slot, page, bar);
      else bulk_load(dst + kRawKs + q * 128 * H, pg + C.ks_off() + static_cast<int64_t>(slot) * 8 * H, 128 * H << per, bar);
    }
    __syncwarp();
  };
  // the first tile, while the others set Q up: their barriers are the CTA's own, and the three warps
  // see them initialised
  if (warp >= kLoadWarp0) {
    asm volatile("barrier.cta.sync 3, %0;" ::"n"(32 * kLoadWarps) : "memory");
    page_next = lookup(0);
    load_tile(0, 0);                                       // (a tile's copies take a warp up to 800 clocks to issue: the others after the barrier)
  }

  // ---- visibility of this thread's row
  int my_vis = 0;
  if (warp < kRowWarps && row / kGqa < tok_n) {
    const int t = tok_first + row / kGqa;
    my_vis = p.steps ? max(0, min(__ldcg(p.steps + t), vis0)) : max(0, vis0 + t - tok0);
  }
  // ---- Q rows of this map -> fp16 with a power of two per row, swizzled K-major: half a warp
  // takes a row at a time (8 elements a lane); every load goes out ahead of the first use (one row after
  // the other took 3.2 us of a unit's 10.5 beside its tiles)
  if (warp < kIssueWarp) {
    constexpr int kPer = kRows / (2 * kIssueWarp);
    const int sub = lane >> 4, l16 = lane & 15;
    uint4 qa[kPer], qb[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = 2 * (warp + kIssueWarp * j) + sub;
      qa[j] = qb[j] = make_uint4(0, 0, 0, 0);
      if (r / kGqa < tok_n) {
        const int64_t e0 = (static_cast<int64_t>(tok_first + r / kGqa) * HQ + g * kGqa + r % kGqa) * kD + 128 * map + 8 * l16;
        const uint4* src = p.q_f32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(p.q) + e0)
                                   : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + e0);
        qa[j] = __ldcg(src);
        if (p.q_f32) qb[j] = __ldcg(src + 1);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = 2 * (warp + kIssueWarp * j) + sub;
      const uint32_t w[8] = {qa[j].x, qa[j].y, qa[j].z, qa[j].w, qb[j].x, qb[j].y, qb[j].z, qb[j].w};
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = __uint_as_float(p.q_f32 ? w[u] : (u & 1) ? w[u >> 1] & 0xffff0000u : w[u >> 1] << 16);
      float amax = 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) amax = fmaxf(amax, fabsf(x[u]));
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      const int ex = amax > 0.0f ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127 : 0;
      const int sh = max(-113, min(100, 14 - ex));
      const float up = ldexpf(1.0f, sh);
      // above 0 also where the product underflows: a masked score is -inf times it
      if (l16 == 0) fsc[r] = fmaxf(p.sm_scale_log2 * ldexpf(1.0f, -sh), 1.2e-38f);
      uint32_t hv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __half2 h2 = __floats2half2_rn(__fmul_rn(x[2 * u], up), __fmul_rn(x[2 * u + 1], up));
        hv[u] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      const uint32_t at = (l16 >> 3) * 16384 + swz(r, l16 & 7);
      sts128(sb + kQOff + at, hv[0], hv[1], hv[2], hv[3]);
      if (p.q_f32) {                                                   // what fp16 leaves of them
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hv[u]));
          const __half2 l2 = __floats2half2_rn(__fmul_rn(x[2 * u], up) - h.x, __fmul_rn(x[2 * u + 1], up) - h.y);
          hv[u] = *reinterpret_cast<const uint32_t*>(&l2);
        }
        sts128(sb + p.q_lo + at, hv[0], hv[1], hv[2], hv[3]);
      }
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_barrier();          // barriers, tensor memory and Q of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  float* const block = p.s.rows + (static_cast<int64_t>(unit) * 2 + rank) * kRows * kDiffRow;   // this CTA's partial rows

  if (warp < kRowWarps) {
    // ================================================================ rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float my_f = fsc[row];
    const uint32_t p_full0 = map_to(bars + 8 * kBarPFull, 0), s_free0 = map_to(bars + 8 * kBarSFree, 0);
    const uint32_t refs = bars + 8 * (kBarRef + 2 * (warp & 3));
    // the running O of a row: float4 number c at acc[128 c] of the block (128 x 260 floats)
    float l = 0.0f, l_ref = -INFINITY;                                 // l counts relative to 2^l_ref
    bool failed = false;
    for (int i = group; i < n_tiles; i += 2) {
      const uint32_t parity = (i >> 1) & 1;
      if (!wait_soon(bars + 8 * (kBarSFull + group), parity, p.wait_ns) ||
          !wait_soon(bars + 8 * (kBarKsFull + (i & 3)), (i >> 2) & 1, p.wait_ns)) {
        failed = true;
        break;
      }
      tc_fence_after();
      float sc[kTileN];
      tmem_ld128(tmem + lane_base, sc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(s_free0);
      // scores, unscaled (my_f > 0, so the maximum commutes with it)
      const float* ks = ksbuf + 128 * (i % kKsRing);
#pragma unroll
      for (int c = 0; c < kTileN; c += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(ks + c);
        const float2 a = __fmul2_rn(make_float2(k4.x, k4.y), make_float2(sc[c], sc[c + 1]));
        const float2 b = __fmul2_rn(make_float2(k4.z, k4.w), make_float2(sc[c + 2], sc[c + 3]));
        sc[c] = a.x; sc[c + 1] = a.y;
        sc[c + 2] = b.x; sc[c + 3] = b.y;
      }
      const int vis = my_vis - (tile0 + i) * kTileN;                   // cells [0, vis) of the tile
      const unsigned odd = ctl[4 + i % kKsRing];                       // 16-cell groups on a page out of range, cells of large blocks
      if (vis < kTileN || odd) {
#pragma unroll
        for (int c = 0; c < kTileN; ++c)
          if (c >= vis || ((odd >> (8 * (c >> 5) + ((c >> 4) & 1))) & 1)) sc[c] = -INFINITY;
      }
      float mx[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
      for (int c = 4; c < kTileN - 4; c += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], fmaxf(sc[c + 2 * k], sc[c + 2 * k + 1]));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], sc[kTileN - 4 + k]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * my_f + (odd & 0x04040404u ? 3.0f : 0.0f);
      // the row's reference, as the tile before left it
      float m_run = -INFINITY, alpha = 1.0f;
      if (i > 0) {
        if (!wait_soon(refs + 8 * (group ^ 1), ((i - 1) >> 1) & 1, p.wait_ns)) {
          failed = true;
          break;
        }
        m_run = ref[row];
      }
      if (top > m_run + kSlack) {
        alpha = ex2_ftz(m_run - top);                                   // 0 on the first visible tile
        m_run = top;
      }
      ref[row] = m_run;
      __syncwarp();
      if (lane == 0) arrive_local(refs + 8 * group);
      if (l_ref != m_run) {                                            // moved, by this tile or the one before
        l = l_ref > -INFINITY ? l * ex2_ftz(l_ref - m_run) : 0.0f;
        l_ref = m_run;
      }
      const float mu = (m_run == -INFINITY ? 0.0f : m_run) - kLift;
      const float2 f2 = make_float2(my_f, my_f);
      // P(i - 2) has been read
      if (i >= 2 && !wait_soon(bars + 8 * (kBarODone + group), ((i - 2) >> 1) & 1, p.wait_ns)) {
        failed = true;
        break;
      }
      float2 psum[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) psum[k] = make_float2(0.0f, 0.0f);
      const uint32_t pcol = tmem + lane_base + kPCol + kPBuf * group;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const bool big = (odd >> (8 * h + 2)) & 1;                     // 8 P, which counts as P in the sum
        const float off = big ? 3.0f - mu : -mu, one = big ? 0.125f : 1.0f;
        const float2 mu2 = make_float2(off, off), counts = make_float2(one, one);
        uint32_t ph[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 e = __ffma2_rn(make_float2(sc[32 * h + 2 * c], sc[32 * h + 2 * c + 1]), f2, mu2);
          const float2 q = make_float2(ex2_ftz(e.x), ex2_ftz(e.y));
          const __half2 hq = __floats2half2_rn(q.x, q.y);
          psum[c & 3] = __ffma2_rn(q, counts, psum[c & 3]);
          ph[c] = *reinterpret_cast<const uint32_t*>(&hq);
        }
        tmem_st16(pcol + 16 * h, ph);
      }
      psum[0] = __fadd2_rn(__fadd2_rn(psum[0], psum[1]), __fadd2_rn(psum[2], psum[3]));
      l += psum[0].x + psum[0].y;
      // O of the tiles so far: into the running sum at every kChain-th tile (both CTAs), rescaled
      // in place where a reference moved in between
      const bool folds = i > 0 && i % kChain == 0;
      if (folds || (i > 0 && __any_sync(kFull, alpha != 1.0f))) {
        if (!wait_soon(bars + 8 * (kBarODone + (group ^ 1)), ((i - 1) >> 1) & 1, p.wait_ns)) {
          failed = true;
          break;
        }
        tc_fence_after();
        // the running sum is relative to the reference too: both move.  The other group's thread of this row wrote it
        // last, and what came between (P's arrival, perhaps at the other CTA's barrier, and the product's completion)
        // orders it for this CTA's threads only with a fence on either side
        const bool have = i > kChain;
        if (have) asm volatile("fence.acq_rel.cluster;" ::: "memory");
        float4* const acc = reinterpret_cast<float4*>(block) + row;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float o[128];                                                // (the scores are done with)
          tmem_ld128(tmem + lane_base + kOCol + 128 * h, o);
          if (folds) {                                                 // acc = (acc + O) * alpha
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float4 old = have ? acc[128 * (32 * h + c)] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              acc[128 * (32 * h + c)] = make_float4((old.x + o[4 * c]) * alpha, (old.y + o[4 * c + 1]) * alpha,
                                                    (old.z + o[4 * c + 2]) * alpha, (old.w + o[4 * c + 3]) * alpha);
            }
          } else {                                                     // O *= alpha
#pragma unroll
            for (int c = 0; c < 128; ++c) o[c] *= alpha;
#pragma unroll
            for (int c = 0; c < 128; c += 32) tmem_st32(tmem + lane_base + kOCol + 128 * h + c, o + c);
            if (have) {
#pragma unroll 4
              for (int c = 0; c < 32; ++c) {
                const float4 old = acc[128 * (32 * h + c)];
                acc[128 * (32 * h + c)] = make_float4(old.x * alpha, old.y * alpha, old.z * alpha, old.w * alpha);
              }
            }
          }
        }
        if (folds || have) asm volatile("fence.acq_rel.cluster;" ::: "memory");
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(p_full0 + 8 * group);
    }
    if (!failed && !wait_soon(bars + 8 * (kBarODone + ((n_tiles - 1) & 1)), ((n_tiles - 1) >> 1) & 1, p.wait_ns)) failed = true;
    if (failed) ctl[1] = 1;
    // PV of the last tile is done in both CTAs (one commit covers the pair), and with it every
    // read of this CTA's operand tiles; past the barrier the last reference is known
    const bool stop = rows_any(failed);
    if (!stop) {
      tc_fence_after();
      const float m_run = ref[row];
      sums[group * kRows + row] = l_ref > -INFINITY ? l * exp2f(l_ref - m_run) : 0.0f;
      float* rowbuf = reinterpret_cast<float*>(smem + kQOff);          // [128][256] fp32, rotated by 4 * row
      const bool have = n_tiles > kChain;
      const float4* const acc = reinterpret_cast<const float4*>(block) + row;
#pragma unroll 1
      for (int h = 4 * group; h < 4 * group + 4; ++h) {                // 128 of the dims to a group
        float o[32];
        tmem_ld32(tmem + lane_base + kOCol + 32 * h, o);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float4 x = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          if (have) {
            const float4 old = acc[128 * (8 * h + c)];
            x.x += old.x; x.y += old.y; x.z += old.z; x.w += old.w;
          }
          *reinterpret_cast<float4*>(rowbuf + row * 256 + ((32 * h + 4 * c + 4 * row) & 255)) =
              make_float4(x.x, x.z, x.y, x.w);                 // (dims 1 and 2 of each four are swapped)
        }
      }
      tc_fence_before();
      rows_barrier();                                                  // rows and sums written, running sums read
      if (group == 0 && row / kGqa < tok_n) {
        block[row * kDiffRow + 256] = m_run - kLift;                   // o and l are relative to 2^(m - kLift)
        block[row * kDiffRow + 257] = sums[row] + sums[kRows + row];
      }
      for (int r = warp; r < kGqa * tok_n; r += kRowWarps) {
        float4* dst = reinterpret_cast<float4*>(block + r * kDiffRow);
        dst[lane] = *reinterpret_cast<const float4*>(rowbuf + r * 256 + ((4 * lane + 4 * r) & 255));
        dst[32 + lane] = *reinterpret_cast<const float4*>(rowbuf + r * 256 + ((128 + 4 * lane + 4 * r) & 255));
      }
    } else if (group == 0 && row / kGqa < tok_n) {                     // nothing to join of a unit that failed
      block[row * kDiffRow + 256] = -INFINITY;
      block[row * kDiffRow + 257] = 0.0f;
    }
  } else if (warp < kIssueWarp) {
    // ================================================================ conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    const int t = tid & 127;
    const bool is_v = warp >= kVConvWarp0;
    // K: cell 64 rank + (t & 63), dims [64 (t >> 6), +64); V: cell t, blocks 4 rank .. 4 rank + 3.
    // The copies put 16-byte unit u of a row at u ^ (row & 7) (128-byte swizzle).
    const int kcell = t & 63, kchunk = t >> 6;
    const uint32_t full0 = map_to(bars + 8 * (is_v ? kBarVFull : kBarKFull), 0);
    const uint32_t kraw = (kcell >> 4) * 2048 + (kcell & 15) * 128;
    const uint32_t vraw = kRawV + (t >> 4) * 2048 + (t & 15) * 128;
    const uint32_t ksraw = kRawKs + (t >> 4) * 128 * C.H + ((t & 15) * C.H + g) * 8 + 4 * map;
    const uint32_t vsraw = kRawKs + 1024 * C.H + (t >> 4) * 256 * C.H + ((t & 15) * C.H + g) * 16;     // a cell's eight V scales
    // a tile's buffers are free once the product of tile i - 2 has read them
    const uint32_t freed = bars + 8 * (is_v ? kBarODone : kBarSFull);
    int stage = 0;
    uint32_t raw_phase = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i & 1;
      const uint32_t raw = sb + kRawOff + stage * p.stage_bytes;
      if (!wait_soon(bars + 8 * (kBarRawFull + stage), raw_phase, p.wait_ns)) { ctl[1] = 1; break; }
      const int valid = ctl[12 + stage];                   // the tile's 16-cell groups that were copied; bits 8..15: on a bad page
      const bool seen = (valid >> (t >> 4)) & 1 && (tile0 + i) * kTileN + t < limit;   // cell t is copied and some row sees it
      if (!is_v) {
        uint4 kw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) kw[u] = lds128(raw + kraw + (((4 * kchunk + u) ^ (kcell & 7)) << 4));
        float ksc;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ksc) : "r"(raw + ksraw));
        const uint4 vd = lds128(raw + vsraw);
        const bool big = __any_sync(kFull, seen && big_blocks(vd));
        if (i >= 2 && !wait_soon(freed + 8 * buf, ((i - 2) >> 1) & 1, p.wait_ns)) { ctl[1] = 1; break; }
        __syncwarp();
        if (lane == 0) arrive_local(bars + 8 * (kBarRawEmpty + stage));
        const uint32_t dst = sb + kKOff + buf * kKBuf + kchunk * 8192;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 w = kw[u];
          uint32_t h[8];
          i8x4_to_f16(w.x, h[0], h[1]);
          i8x4_to_f16(w.y, h[2], h[3]);
          i8x4_to_f16(w.z, h[4], h[5]);
          i8x4_to_f16(w.w, h[6], h[7]);
          sts128(dst + swz(kcell, 2 * u), h[0], h[1], h[2], h[3]);
          sts128(dst + swz(kcell, 2 * u + 1), h[4], h[5], h[6], h[7]);
        }
        ksbuf[128 * (i % kKsRing) + t] = ksc;
        if (lane == 0) {
          reinterpret_cast<volatile uint8_t*>(ctl + 4 + i % kKsRing)[t >> 5] = static_cast<uint8_t>(((valid >> 8) >> (2 * (t >> 5)) & 3) | (big ? 4 : 0));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          arrive_local(bars + 8 * (kBarKsFull + (i & 3)));
          arrive_cluster(full0 + 8 * buf);
        }
      } else {
        const uint32_t dst = sb + kVOff + buf * kVBuf;
        // a cell that was not copied, or that nobody sees, counts with V = 0 (its P is 0, its bytes are anything)
        const uint4 all = lds128(raw + vsraw);
        uint32_t vd[2] = {rank ? all.z : all.x, rank ? all.w : all.y};
        if (__any_sync(kFull, seen && big_blocks(all))) vd[0] = eighth_of(vd[0]), vd[1] = eighth_of(vd[1]);
        uint4 vw[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) vw[b] = lds128(raw + vraw + (((4 * rank + b) ^ (t & 7)) << 4));
        if (!seen) vd[0] = vd[1] = 0;
        if (i >= 2 && !wait_soon(freed + 8 * buf, ((i - 2) >> 1) & 1, p.wait_ns)) { ctl[1] = 1; break; }
        __syncwarp();
        if (lane == 0) arrive_local(bars + 8 * (kBarRawEmpty + stage));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const __half dh = __ushort_as_half(static_cast<unsigned short>(vd[b >> 1] >> (16 * (b & 1))));
          const __half2 d2 = __halves2half2(dh, dh);
          uint32_t lo[8], hi[8];                           // dims 0..15 of the block, and 16..31
          nib_word(vw[b].x, d2, lo, hi);
          nib_word(vw[b].y, d2, lo + 2, hi + 2);
          nib_word(vw[b].z, d2, lo + 4, hi + 4);
          nib_word(vw[b].w, d2, lo + 6, hi + 6);
          const uint32_t at = dst + (b >> 1) * kVAtom;     // 64 dims an atom
          const int u0 = 4 * (b & 1);
          sts128(at + swz(t, u0), lo[0], lo[1], lo[2], lo[3]);
          sts128(at + swz(t, u0 + 1), lo[4], lo[5], lo[6], lo[7]);
          sts128(at + swz(t, u0 + 2), hi[0], hi[1], hi[2], hi[3]);
          sts128(at + swz(t, u0 + 3), hi[4], hi[5], hi[6], hi[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cluster(full0 + 8 * buf);
      }
      if (++stage == p.stages) {
        stage = 0;
        raw_phase ^= 1;
      }
    }
  } else {
    // ================================================================ issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    // The whole warp runs the loop and one elected lane executes the products: with the
    // control flow uniform the descriptors live in uniform registers
    if (__shfl_sync(kFull, warp, 0) == kIssueWarp) {
      if (rank == 0) {
        constexpr uint32_t idS = idesc_f16(256, 128, false, false);
        constexpr uint32_t idO = idesc_f16(256, 256, false, true);
        const uint32_t tm = __shfl_sync(kFull, tmem, 0);
        const uint64_t dq0 = smem_desc(sb + kQOff, 16, 1024);
        const uint64_t dl0 = smem_desc(sb + p.q_lo, 16, 1024);
        const uint64_t dk0 = smem_desc(sb + kKOff, 16, 1024);
        const uint64_t dv0 = smem_desc(sb + kVOff, kVAtom, 1024);
        const bool leader = elect_one();
        auto qk = [&](int buf) {                           // S = Q K^T
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk & 3) * 32;
            mma_pair(tm, dq0 + (((kk >> 2) * 16384 + off) >> 4), dk0 + ((buf * kKBuf + (kk >> 2) * 8192 + off) >> 4), idS, kk ? 1u : 0u);
          }
          if (p.q_f32) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk & 3) * 32;
              mma_pair(tm, dl0 + (((kk >> 2) * 16384 + off) >> 4), dk0 + ((buf * kKBuf + (kk >> 2) * 8192 + off) >> 4), idS, 1u);
            }
          }
          commit_both(bars + 8 * (kBarSFull + buf));
        };
        // Whatever is ready goes out: S(si) once S(si - 1) is in the rows' registers (so that a group finds its next
        // tile scored when it is done with this one), O(oi) once P and V are there.  A fixed order of the two
        // holds one back for the other
        auto test = [&](int bar, uint32_t parity) -> bool { return __all_sync(kFull, mbar_test(bars + 8 * bar, parity)) != 0; };
        bool ok = true;
        uint64_t since = 0;                                // of a turn with nothing ready; 0: the last one had
        for (int si = 0, oi = 0; oi < n_tiles;) {
          bool idle = true;
          if (si < n_tiles && test(kBarKFull + (si & 1), (si >> 1) & 1) && (si == 0 || test(kBarSFree, (si - 1) & 1))) {
            tc_fence_after();
            if (leader) qk(si & 1);
            ++si;
            idle = false;
          }
          const int buf = oi & 1;
          const uint32_t parity = (oi >> 1) & 1;
          if (oi < si && test(kBarVFull + buf, parity) && test(kBarPFull + buf, parity)) {
            tc_fence_after();
            if (leader) {
              const uint32_t more = oi % kChain != 0 ? 1u : 0u;   // O of this chain so far is kept
              const uint32_t pa = tm + kPCol + kPBuf * buf;
              const uint64_t v0 = dv0 + ((buf * kVBuf) >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)                 // 16 cells = 8 columns of fp16 pairs
                mma_pair_ta(tm + kOCol, pa + 8 * kk, v0 + ((kk * 2048) >> 4), idO, kk ? 1u : more);
              commit_both(bars + 8 * (kBarODone + buf));
            }
            ++oi;
            idle = false;
          }
          if (!idle) {
            since = 0;
            continue;
          }
          const uint64_t now = __shfl_sync(kFull, global_ns(), 0);
          if (since == 0) since = now;
          if (p.wait_ns < 1000u || now - since >= p.wait_ns) { ok = false; break; }
          (void)mbar_try(bars + 8 * (kBarPFull + buf), parity, 100u);
          __syncwarp();
        }
        if (!ok) ctl[1] = 1;
        // all of this warp's products, waited for below (after a failure too)
        if (leader) commit_both(bars + 8 * kBarDrain);
      }
    } else {
      // ============================================================== copies
      int i = 1, stage = 1 % p.stages;
      uint32_t phase = p.stages == 1 ? 0 : 1;              // of the stage's last use
      for (; i < n_tiles; ++i) {
        if (i >= p.stages && !__all_sync(kFull, wait_soon(bars + 8 * (kBarRawEmpty + stage), phase, p.wait_ns))) { ctl[1] = 1; break; }
        load_tile(i, stage);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // no copy is in flight past here (after a failure too): the last tiles' stages
      for (int j = max(0, i - p.stages); j < i; ++j)
        (void)mbar_wait(bars + 8 * (kBarRawFull + j % p.stages), (j / p.stages) & 1, kWaitDefaultNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // The commits arrive at the barriers of both CTAs, and each CTA waits for its own copies of the
  // last ones: shared memory that an arrival is still on its way to must not be given to the
  // next CTA.  (The row warps have waited for every S and the last O.)
  if (warp == kIssueWarp) {
    if (n_tiles > 1 && !ctl[1])
      (void)mbar_wait(bars + 8 * (kBarODone + (n_tiles & 1)), ((n_tiles - 2) >> 1) & 1, kWaitDefaultNs);
    (void)mbar_wait(bars + 8 * kBarDrain, 0, kWaitDefaultNs);
    __syncwarp();
  }
  if (tid == 0 && ctl[1]) record_status(p.status, K8V4_ECUDA);
  cluster_barrier();          // no product, commit or arrival of the pair is in flight
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host side
// Set-up of the pair kernel on the current device: its shared memory, its registers at launch (the
// split hands out that many) and the CTA pairs that the device runs at a time.  Kept once it has
// worked; a failure is not, and the next call tries again.
std::mutex g_pairs_mu;
int g_pairs[64];
int device_pairs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(g_pairs_mu);
  if (g_pairs[dev] > 0) return g_pairs[dev];
  cudaFuncAttributes fa;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  if (cudaFuncGetAttributes(&fa, diff_pair_kernel) != cudaSuccess ||
      fa.numRegs * 5 < 2 * kRowRegs + 2 * kConvRegs + kIssueRegs ||
      cudaFuncSetAttribute(diff_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&pairs, diff_pair_kernel, &cfg) != cudaSuccess || pairs < 1) {
    cudaGetLastError();                   // clear the error state that the failed call left
    return 0;
  }
  return g_pairs[dev] = pairs;
}
// A tensor map of a cache's K or V rows as the decode's, with boxes of `box` cells
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}
bool encode_rows(CUtensorMap* m, const CacheView& C, int64_t run_off, int row_bytes, int box) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(C.H), static_cast<cuuint64_t>(C.P),
                              static_cast<cuuint64_t>(C.n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(row_bytes) * C.H,
                                 static_cast<cuuint64_t>(C.page_bytes)};
  const cuuint32_t shape[4] = {128, 1, static_cast<cuuint32_t>(box), 1}, one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, C.pages + run_off, dims, strides, shape, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// the pairs that a workspace and its schedule are sized for: of the device's SMs, the same whether or
// not the set-up has worked yet
int planned_pairs(int num_sms) { return std::max(1, std::min(num_sms / 2, kDiffMostPairs)); }

}  // namespace

size_t diff_ws_bytes(const CacheView& C, int n_seqs, int n_tok, int max_seq_len, int num_sms) {
  return place(nullptr, nullptr, n_seqs, n_tok, max_seq_len, C.H, planned_pairs(num_sms), num_sms);
}

int launch_diff(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* offsets, int n_tok,
                const int32_t* pt, int64_t max_pages, const int32_t* lens, const int32_t* steps, int n_seqs,
                int max_seq_len, float sm_scale, const k8v4_diff& diff, void* out, void* ws) {
  if (device_pairs() < 1) return K8V4_ECUDA;
  const int pairs = planned_pairs(L.num_sms);
  ScheduleParams sp;
  place(&sp.s, static_cast<uint8_t*>(ws), n_seqs, n_tok, max_seq_len, C.H, pairs, L.num_sms);
  sp.d = diff;
  sp.offsets = offsets;
  sp.lens = lens;
  sp.steps = steps;
  sp.n_seqs = n_seqs;
  sp.n_tok = n_tok;
  sp.max_seq_len = max_seq_len;
  sp.H = C.H;
  sp.pairs = pairs;
  sp.most = most_units(n_seqs, n_tok, max_seq_len, C.H, pairs);
  sp.more = more_units(most_tiles(n_seqs, n_tok) * 2 * C.H, pairs, n_seqs, n_tok);
  sp.most_rows = most_rows(n_seqs, n_tok);
  sp.status = L.status;
  int rc = launch_behind(L, diff_schedule_kernel, dim3(1), dim3(1024), sp);
  if (rc) return rc;
  rc = launch_diff_split(L, C, q, q_dtype, pt, max_pages, sp.s.row_vis, DiffQueries{sp.s.row_seq, sp.s.row_tok, sp.s.head + 1}, 0,
                         max_seq_len, sm_scale, sp.s.pieces);
  if (rc) return rc;
  PairParams p;
  p.C = C;
  p.q = q;
  p.q_f32 = q_dtype == K8V4_F32;
  p.pt = pt;
  p.max_pages = max_pages;
  p.steps = steps;
  p.s = sp.s;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.status = L.status;
  p.wait_ns = wait_limit_ns() ? wait_limit_ns() : kWaitDefaultNs;
  p.page_div = FastDiv(static_cast<uint32_t>(C.P));
  p.stages = raw_stages(C.H, p.q_f32);
  p.stage_bytes = raw_bytes(C.H);
  p.q_lo = p.q_f32 ? kRawOff + p.stages * p.stage_bytes : kQOff;
  p.box_shift = C.P % 64 == 0 ? 6 : C.P % 32 == 0 ? 5 : 4;
  CUtensorMap mk, mv;
  if (!encode_rows(&mk, C, 0, 256, 1 << p.box_shift) || !encode_rows(&mv, C, C.v_off(), 128, 1 << p.box_shift)) return K8V4_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * sp.most));                // below 2^25 with n_tok < 2^24, n_seqs < 2^16
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRawOff + p.stages * p.stage_bytes + (p.q_f32 ? kQBytes : 0);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, diff_pair_kernel, mk, mv, p) != cudaSuccess) return K8V4_ECUDA;
  if (cudaGetLastError() != cudaSuccess) return K8V4_ECUDA;
  DiffRagged r;
  r.lambdas = sp.s.lambdas;
  r.tok_tile = sp.s.tok_tile;
  r.tiles = reinterpret_cast<const int32_t*>(sp.s.tiles);
  // few token tiles: their rows have tens of ranges each, and a row gets four warps
  const bool few = most_tiles(n_seqs, n_tok) * 2 * C.H < pairs;
  return launch_diff_combine_ragged(L, sp.s.rows, r, sp.s.pieces, sp.s.row_vis, n_tok, C.H, few, diff, out);
}

}  // namespace k8v4
