// ar_w4_matvec and ar_w4_matvec_experts: checks and the launch shape.  The
// kernels (w4_matvec.cuh) are compiled in w4_<scale type>_<zero points: z or
// n><experts: e or d>.cu.
#include <cmath>
#include <mutex>

#include "w4_matvec.cuh"

namespace arn {

// Row tiles 1 or 2, column tiles 1 or 2, groups of 32, 64 or 128.
W4Kernel w4_kernel_f32_nd(int r, int nt, int group);
W4Kernel w4_kernel_f32_ne(int r, int nt, int group);
W4Kernel w4_kernel_f32_zd(int r, int nt, int group);
W4Kernel w4_kernel_f32_ze(int r, int nt, int group);
W4Kernel w4_kernel_bf16_nd(int r, int nt, int group);
W4Kernel w4_kernel_bf16_ne(int r, int nt, int group);
W4Kernel w4_kernel_bf16_zd(int r, int nt, int group);
W4Kernel w4_kernel_bf16_ze(int r, int nt, int group);
W4Kernel w4_kernel_f16_nd(int r, int nt, int group);
W4Kernel w4_kernel_f16_ne(int r, int nt, int group);
W4Kernel w4_kernel_f16_zd(int r, int nt, int group);
W4Kernel w4_kernel_f16_ze(int r, int nt, int group);

static W4Kernel w4_kernel(int type, bool zeros, bool experts, int r, int nt, int group) {
  using Pick = W4Kernel (*)(int, int, int);
  static const Pick picks[3][2][2] = {
      {{w4_kernel_f32_nd, w4_kernel_f32_ne}, {w4_kernel_f32_zd, w4_kernel_f32_ze}},
      {{w4_kernel_bf16_nd, w4_kernel_bf16_ne}, {w4_kernel_bf16_zd, w4_kernel_bf16_ze}},
      {{w4_kernel_f16_nd, w4_kernel_f16_ne}, {w4_kernel_f16_zd, w4_kernel_f16_ze}}};
  return picks[type][zeros ? 1 : 0][experts ? 1 : 0](r, nt, group);
}

// Every kernel may use all of an SM's shared memory; set once per device by
// the first call, which must be outside graph capture (as for the rest of
// the library).
static int allow_shared_memory(int bytes) {
  static std::mutex mu;
  static bool done[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return AR_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return AR_OK;
  for (int type = AR_TYPE_F32; type <= AR_TYPE_F16; ++type)
    for (int i = 0; i < 16; ++i)
      for (int group = 32; group <= 128; group *= 2) {
        if (group == 32 && (i & 4)) continue;  // one row tile
        const W4Kernel kern = w4_kernel(type, i & 1, i & 2, i & 4 ? 2 : 1, i & 8 ? 2 : 1, group);
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 bytes) != cudaSuccess) {
          cudaGetLastError();
          return AR_ERR_CUDA;
        }
      }
  done[dev] = true;
  return AR_OK;
}

struct W4Plan {
  int r, nt, warps, team, units, phases, phase_units, cols, x_cols;
  int64_t rounds;  // items of a team, about
};

// Lays out shared memory for a plan: the fewest phases (of p->units) with
// which x of a set fits into `most`, and as many columns of x as do (no more
// than the sets could fill); false if not even a unit's fits.
static bool w4_layout(W4Plan *p, int group, int64_t most, bool experts, W4Args *a) {
  const int64_t unit = int64_t{w4_parts(p->r, p->nt, group)} * 256;  // x of a unit's column
  const int64_t tile = int64_t{p->cols} * 16 * p->r * 4;
  const int64_t ring = int64_t{p->warps} * w4_ring_bytes(p->r, p->nt, group);
  const int64_t red = p->team > 1 ? int64_t{2} * p->warps * tile : 0;
  const int64_t ids = experts ? (int64_t{2} * a->pairs + 15) / 16 * 16 : 0;
  const int teams = p->warps / p->team;
  // Sums between phases: as many items a team as 32 KB hold.
  a->phase_rounds = static_cast<int>(32768 / (teams * tile));
  if (a->phase_rounds > p->rounds) a->phase_rounds = static_cast<int>(p->rounds);
  if (a->phase_rounds < 1) a->phase_rounds = 1;
  int64_t room = most - ring - red - ids, acc = 0;  // for x
  p->phases = 1;
  if (p->cols * p->units * unit > room) {
    acc = a->phase_rounds * teams * tile;
    room -= acc;
    const int64_t fit = room < 0 ? 0 : room / (p->cols * unit);
    if (fit < 1) return false;
    p->phases = static_cast<int>((p->units + fit - 1) / fit);
  }
  p->phase_units = (p->units + p->phases - 1) / p->phases;
  const int64_t column = p->phase_units * unit;
  int64_t x_cols = p->phases > 1 ? p->cols : room / column;  // a phase holds one set
  if (x_cols > kW4MaxXCols) x_cols = kW4MaxXCols;
  if (x_cols > a->pairs) x_cols = a->pairs;
  p->x_cols = static_cast<int>(x_cols);
  int64_t at = ring;
  a->xs_offset = static_cast<int>(at);
  at += x_cols * column;
  a->red_offset = static_cast<int>(at);
  at += red;
  a->acc_offset = static_cast<int>(at);
  at += acc;
  a->ids_offset = static_cast<int>(at);
  at += ids;
  a->smem_bytes = static_cast<int>(at);
  return true;
}

// How many of E experts with `pairs` choices have more than n tokens, n < 64,
// if their numbers are Poisson (0 from `end` on: too few to count).
struct Crowds {
  double above[64];
  int end;
  Crowds(int E, double mean) {
    double p = exp(-mean), rest = 1 - p;
    for (end = 0; end < 64 && rest > 1e-3;) {
      above[end] = E * rest;
      p *= mean / ++end;
      rest -= p;
    }
  }
  // Column sets of all experts: one for more than 0, cols, 2 cols, ... tokens.
  double sets(int cols) const {
    double s = 0;
    for (int n = 0; n < end; n += cols) s += above[n];
    return s;
  }
};

// The launch shape: row and column tiles, team, columns of a set and phases
// that minimise an estimate of a CTA's time.
//   - Teams go through their items in rounds.  A round with all warps at work
//     takes in 41 KB/us with one row tile and one column tile; somewhat more
//     with two row tiles where rows are short (32 tokens, 112 experts of 1024
//     x 6144: 76 us against 86 us) and less where they are long (4 tokens, 25
//     of 64 experts of 7168 x 4096, gated: 109 us against 90 us); 27 KB/us
//     with two column tiles (16 x 2048 x 32768: 17.4 us, where one reads the
//     weights twice in 19.9 us).  A last round of few warps is not much
//     faster than their share.
//   - The end of a round costs 2 us, with the joined sums of larger teams 2.6
//     to 3.3 us (1 x 7168 x 7168: 14.4, 11.8, 10.7 and 11.8 us with teams of
//     1, 2, 4 and 8).
//   - x takes 0.021 us a KB to unpack, and 2.2 us each time.  Experts, which
//     seldom have all the columns that a set could, take a few less where
//     that spares the phases (16 tokens of 7168, 8 of 64 experts: 7 columns
//     in 176 us, 8 in 199 us).
// Over 45 shapes the choice is within 2 % of the best shape on average.
static bool w4_plan(int64_t m, bool experts, int group, int64_t most, int sms, W4Args *a,
                    W4Plan *best) {
  double least = 0;
  bool found = false;
  W4Plan p = {};
  p.warps = kW4MaxWarps;
  const int per_row = a->act == AR_ACT_SILU_MUL ? 8 : 16;  // outputs of a row tile
  const double mean = static_cast<double>(a->pairs) / a->E;
  const Crowds crowds(a->E, experts && mean <= 16 ? mean : 0);
  // Two column tiles for experts only where they fill them (64 tokens, 16 an
  // expert, of 4096 x 4096, gated: 54 us against 44 us).
  const int most_nt = m > 8 && (!experts || mean > 16) ? 2 : 1;
  for (p.nt = 1; p.nt <= most_nt; ++p.nt) {
    const int widest = static_cast<int>(m < 8 * p.nt ? m : 8 * p.nt);
    bool whole = false;  // a plan of one phase
    for (p.cols = widest; p.cols > (experts ? widest / 2 : widest - 1) && !whole; --p.cols) {
      const double sets = !experts ? static_cast<double>((m + p.cols - 1) / p.cols)
                          : mean > 16 ? a->E * (mean / p.cols + 0.5) : crowds.sets(p.cols);
      for (p.r = 1; p.r <= (group == 32 ? 1 : 2); ++p.r) {
        const int parts = w4_parts(p.r, p.nt, group), unit_k = parts * kW4PartK;
        p.units = (a->K + unit_k - 1) / unit_k;
        const int64_t blocks = (a->width + per_row * p.r - 1) / (per_row * p.r);
        const int64_t each = static_cast<int64_t>(
            experts ? ceil(sets * blocks / sms) : ceil(blocks / floor(sms / sets)));
        double rate = p.nt == 2 ? 27 : 41;
        if (p.r == 2) rate *= 1.08 / (1 + a->K / 18000.);
        const double item = p.r * p.units * parts / rate;
        // Column sets that a CTA may meet, and their columns.
        const int64_t met = !experts || each == 1 ? 1 : 1 + (each - 1 + blocks - 1) / blocks;
        const double columns = met * (a->pairs / sets);
        for (p.team = 1; p.team <= p.warps; p.team *= 2) {
          const int teams = p.warps / p.team;
          const int64_t rest = each % teams;
          p.rounds = (each + teams - 1) / teams;
          if (!w4_layout(&p, group, most, experts, a)) continue;
          if (p.phases == 1) whole = true;
          double time = (each - rest) * item;
          if (rest > 0) {
            const double share = 1.6 * rest * p.team / p.warps;
            time += rest * item / (share < 1 ? share : 1);
          }
          time += p.rounds * p.phases * (p.team == 1 ? 2 : 2.5 + 0.05 * p.team) +
                  2.2 * p.phases * (columns <= p.x_cols ? 1 : met) + 0.021 * columns * a->K / 512;
          if (!found || time < least) {
            least = time;
            *best = p;
            found = true;
          }
        }
      }
    }
  }
  if (found) {
    a->units = best->units;
    w4_layout(best, group, most, experts, a);
  }
  return found;
}

static int run_w4(const void *x, int x_per_pair, const int32_t *ids, int64_t m, int k, const void *q,
                  const void *scales, int scales_type, const void *zeros, int first, int E, int64_t N,
                  int64_t K, int group, int act, void *out, bool experts, void *stream) {
  const int size = type_size(scales_type);
  if (m < 0 || k < 1 || first < 0 || E < 1 || N < 1 || K < 1 || size == 0 ||
      (group != 32 && group != 64 && group != 128) || (act != AR_ACT_NONE && act != AR_ACT_SILU_MUL) ||
      (x_per_pair != 0 && x_per_pair != 1))
    return AR_ERR_ARG;
  if (K % group != 0 || (act == AR_ACT_SILU_MUL && N % 2 != 0)) return AR_ERR_ARG;
  if (E > AR_MAX_EXPERTS || k > AR_MAX_TOPK || K > AR_MATVEC_MAX_K || N > AR_MATVEC_MAX_N ||
      m > (experts ? AR_MATVEC_MAX_PAIRS / k : AR_MATVEC_MAX_ROWS))
    return AR_ERR_UNSUPPORTED;
  if (m == 0) return AR_OK;
  if (!x || !q || !scales || !out || (experts && !ids)) return AR_ERR_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned_to(out, 2) || !aligned_to(ids, 4))
    return AR_ERR_ALIGN;
  const int64_t pairs = m * k, ng = K / group;
  const int64_t width = act == AR_ACT_SILU_MUL ? N / 2 : N;
  const Range o = range_of(out, pairs * width * 2);
  if (overlap(o, range_of(x, (x_per_pair ? pairs : m) * K * 2)) ||
      overlap(o, range_of(ids, ids ? pairs * 4 : 0)) || overlap(o, range_of(q, E * N * (K / 2))) ||
      overlap(o, range_of(scales, E * N * ng * size)) ||
      overlap(o, range_of(zeros, zeros ? E * N * ng : 0)))
    return AR_ERR_ALIAS;
  int st;
  DeviceState *d = current_device(&st);
  if (!d) return st;
  // Dynamic shared memory beside the kernels' own (the experts' tables).
  const int64_t most = d->smem_optin - 8192;
  st = allow_shared_memory(static_cast<int>(most));
  if (st != AR_OK) return st;
  W4Args a = {};
  a.x = static_cast<const uint4 *>(x);
  a.ids = ids;
  a.q = static_cast<const uint8_t *>(q);
  a.scales = static_cast<const uint8_t *>(scales);
  a.zeros = static_cast<const uint8_t *>(zeros);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.pairs = static_cast<int>(pairs);
  a.k = x_per_pair ? 1 : k;
  a.first = first;
  // No int32 behind the largest: an id that wraps around is no expert here.
  const int64_t numbered = int64_t{INT32_MAX} - first + 1;
  a.E = static_cast<int>(E < numbered ? E : numbered);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.ng = static_cast<int>(ng);
  a.scale_count = E * N * ng;
  a.width = static_cast<int>(width);
  a.act = act;
  a.status = d->status;

  W4Plan p;
  if (!w4_plan(m, experts, group, most, d->sms, &a, &p)) return AR_ERR_UNSUPPORTED;
  a.cols = p.cols;
  a.x_cols = p.x_cols;
  a.warps = p.warps;
  a.team = p.team;
  a.phase_units = p.phase_units;
  a.wait_limit_ns = kWaitLimitNs;
  const int64_t per_block = (act == AR_ACT_SILU_MUL ? 8 : 16) * p.r;
  a.row_blocks = static_cast<int>((width + per_block - 1) / per_block);
  int64_t ctas;
  if (experts) {  // at most as many as items: each column set has an expert of its own or is full
    ctas = E + pairs / p.cols;
    if (ctas > pairs) ctas = pairs;
    ctas *= a.row_blocks;
    if (ctas > d->sms) ctas = d->sms;
  } else {  // at most eight sets
    const int64_t sets = (m + p.cols - 1) / p.cols;
    a.set_ctas = static_cast<int>(d->sms / sets < a.row_blocks ? d->sms / sets : a.row_blocks);
    ctas = sets * a.set_ctas;
  }
  const W4Kernel kern = w4_kernel(scales_type, zeros != nullptr, experts, p.r, p.nt, group);
  return launch_pdl(kern, a, ctas, p.warps * 32, static_cast<size_t>(a.smem_bytes), 1,
                    static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}

}  // namespace arn

using namespace arn;

extern "C" {

int ar_w4_matvec(const void *x, const void *q, const void *scales, int scales_type,
                 const void *zeros, int64_t m, int64_t N, int64_t K, int group, int act, void *out,
                 void *stream) {
  return run_w4(x, 0, nullptr, m, 1, q, scales, scales_type, zeros, 0, 1, N, K, group, act, out, false,
                stream);
}

int ar_w4_matvec_experts(const void *x, int x_per_pair, const int32_t *ids, int64_t m, int k,
                         const void *q, const void *scales, int scales_type, const void *zeros,
                         int first, int E, int64_t N, int64_t K, int group, int act, void *out,
                         void *stream) {
  return run_w4(x, x_per_pair, ids, m, k, q, scales, scales_type, zeros, first, E, N, K, group, act,
                out, true, stream);
}

}  // extern "C"
