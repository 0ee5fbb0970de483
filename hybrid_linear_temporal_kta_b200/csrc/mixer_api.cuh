// mixer_api.cuh -- host side of the rotary, short-convolution and state-space entry points
// (declared in include/kta.h): argument checks, work decomposition, launches. Included by
// kta_api.cu, whose helpers it uses. Scratch is the caller's: a captured graph then replays on
// memory that no other call or graph shares.

namespace {

constexpr size_t kMixerAlign = 256;

size_t mixer_round(size_t n) { return (n + kMixerAlign - 1) / kMixerAlign * kMixerAlign; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Inputs and outputs of one call: null and alignment checks, then no output may share bytes with
// any other tensor of the call.
struct Span {
  const void* p;
  size_t bytes;
  bool out, required;
  const char* name;
  unsigned align = 16;
};

kta_status check_spans(const Span* v, int n) {
  for (int i = 0; i < n; ++i) {
    if (!v[i].p) {
      if (v[i].required) return fail(KTA_ERR_INVALID_ARG, "%s must not be null", v[i].name);
      continue;
    }
    if (reinterpret_cast<uintptr_t>(v[i].p) % v[i].align)
      return fail(KTA_ERR_ALIGNMENT, "%s is not %u-byte aligned", v[i].name, v[i].align);
  }
  for (int i = 0; i < n; ++i)
    if (v[i].out)
      for (int j = 0; j < n; ++j)
        if (j != i && overlaps(v[i].p, v[i].bytes, v[j].p, v[j].bytes))
          return fail(KTA_ERR_INVALID_ARG, "%s overlaps %s", v[i].name, v[j].name);
  return KTA_OK;
}

kta_status check_grid(long long blocks) {
  if (blocks > 0x7fffffffLL) return fail(KTA_ERR_UNSUPPORTED, "too many blocks (%lld)", blocks);
  return KTA_OK;
}

// Launches a kernel that the one before it on the stream (of the same call) may start early: it waits
// for that one's end itself, where it needs its results. The scan's backward gains 4 % (307 -> 295 us at
// 2 x 2,048 x 2,048 x 16); its forward lost as much on short inputs and launches in order.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ------------------------------------------------------------------------- rotary

template <typename T>
kta_status launch_rope(const kta::RopeParams& p, int W, dim3 grid, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(p.tt) * (p.rot / 2) * sizeof(float2);
  TraceScope ts("rope", st);
  auto kern = W == 0 ? kta::rope_kernel<T, 0> : W == 1 ? kta::rope_kernel<T, 1> : W == 2 ? kta::rope_kernel<T, 2>
                                                                                   : kta::rope_kernel<T, 4>;
  if constexpr (sizeof(T) == 2)
    if (W == 8) kern = kta::rope_kernel<T, 8>;
  kern<<<grid, kta::ROPE_THREADS, smem, st>>>(p);
  KTA_CUDA(cudaGetLastError());
  return KTA_OK;
}

kta_status rope_common(const kta_rope* cfg, const void* x, void* o, const void* x2, void* o2,
                       const kta_shape& s, int H, int ld_heads, int H2, int ld_heads2, float sgn,
                       void* stream) {
  kta_status r;
  if (!cfg) return fail(KTA_ERR_INVALID_ARG, "null rotary description");
  if ((r = check_shape(s)) || (r = check_heads(H, ld_heads, s)) || (r = check_ptrs({x, o}))) return r;
  const bool two = x2 || o2;
  if (two && ((r = check_heads(H2, ld_heads2, s)) || (r = check_ptrs({x2, o2})))) return r;
  if (!cfg->freqs || (reinterpret_cast<uintptr_t>(cfg->freqs) & 7))
    return fail(cfg->freqs ? KTA_ERR_ALIGNMENT : KTA_ERR_INVALID_ARG, "freqs must be 8-byte aligned, not null");
  if (reinterpret_cast<uintptr_t>(cfg->pos) & 7) return fail(KTA_ERR_ALIGNMENT, "pos must be 8-byte aligned");
  if (cfg->n_axes < 1 || cfg->n_axes > kta::ROPE_MAX_AXES)
    return fail(KTA_ERR_INVALID_ARG, "n_axes must be in [1, %d]", kta::ROPE_MAX_AXES);
  if (!cfg->pos && cfg->n_axes > 1) return fail(KTA_ERR_INVALID_ARG, "several axes need positions");
  if (cfg->begin < 0 || cfg->begin % 2) return fail(KTA_ERR_INVALID_ARG, "begin must be even and >= 0");
  if (!std::isfinite(cfg->mscale)) return fail(KTA_ERR_INVALID_ARG, "mscale must be finite");
  kta::RopeParams p{};
  long long rot = 0;
  for (int a = 0; a < cfg->n_axes; ++a) {
    if (cfg->dims[a] < 2 || cfg->dims[a] % 2 || cfg->dims[a] > s.d)
      return fail(KTA_ERR_INVALID_ARG, "dims of axis %d must be even and in [2, d]", a);
    rot += cfg->dims[a];
    p.pair_end[a] = static_cast<int>(rot / 2);
  }
  if (cfg->begin + rot > s.d) return fail(KTA_ERR_INVALID_ARG, "begin + the axes' dims exceed d");
  const size_t es = elem_size(s.dtype);
  const long long N = static_cast<long long>(s.F) * s.P, rows = s.B * N;
  const void* xs[2] = {x, x2};
  void* os[2] = {o, o2};
  const int Hs[2] = {H, two ? H2 : 0}, lds[2] = {ld_heads, two ? ld_heads2 : 0};
  for (int w = 0; w < 2; ++w) {
    p.x[w] = xs[w];
    p.o[w] = os[w];
    p.H[w] = Hs[w];
    p.ld[w] = static_cast<long long>(lds[w]) * s.d;
    p.copy[w] = xs[w] != os[w] && rot < s.d;
  }
  // the heads of a call end before the row does: the last row's tail belongs to no head of it
  auto bytes = [&](int w) { return ((rows - 1) * p.ld[w] + static_cast<long long>(Hs[w]) * s.d) * es; };
  auto clash = [&](const void* a, int wa, const void* b, int wb) {
    if (!a || !b || !overlaps(a, bytes(wa), b, bytes(wb))) return false;
    // head ranges of one tensor: rows of the same stride whose heads do not meet
    if (p.ld[wa] != p.ld[wb]) return true;
    const long long row = p.ld[wa] * static_cast<long long>(es);
    long long off = (static_cast<const char*>(b) - static_cast<const char*>(a)) % row;
    if (off < 0) off += row;
    const long long na = static_cast<long long>(Hs[wa]) * s.d * es, nb = static_cast<long long>(Hs[wb]) * s.d * es;
    return !(off >= na && off + nb <= row);
  };
  // angles are read again while heads are written
  const size_t npos = 8 * static_cast<size_t>(cfg->pos_per_seq ? rows : N) * cfg->n_axes, nfreq = 4 * static_cast<size_t>(rot);
  for (int w = 0; w < 2; ++w)
    if (overlaps(os[w], bytes(w), cfg->pos, npos) || overlaps(os[w], bytes(w), cfg->freqs, nfreq))
      return fail(KTA_ERR_INVALID_ARG, "an output overlaps pos or freqs");
  if ((o != x && clash(o, 0, x, 0)) ||
      (two && ((o2 != x2 && clash(o2, 1, x2, 1)) || clash(o, 0, x2, 1) || clash(o2, 1, x, 0) ||
               clash(o, 0, o2, 1))))
    return fail(KTA_ERR_INVALID_ARG, "an output overlaps another tensor (only o = x and o2 = x2 may coincide)");
  p.rows = rows;
  p.N = static_cast<int>(N);
  p.d = s.d;
  p.begin = cfg->begin;
  p.rot = static_cast<int>(rot);
  p.n_axes = cfg->n_axes;
  p.pos = reinterpret_cast<const long long*>(cfg->pos);
  p.pos_seq = cfg->pos_per_seq ? N * cfg->n_axes : 0;
  p.pos0 = cfg->pos0;
  p.freqs = cfg->freqs;
  p.mscale = cfg->mscale;
  p.sgn = sgn;
  // half layout: partners that lie together, up to a whole piece
  const int V = static_cast<int>(16 / es);
  int W = 0;
  if (!cfg->interleaved) {
    auto fits = [&](int v) {
      if (cfg->begin % v) return false;
      for (int a = 0; a < cfg->n_axes; ++a)
        if (cfg->dims[a] / 2 % v) return false;
      return true;
    };
    for (W = V; W > 1 && !fits(W);) W /= 2;
  }
  p.n_items = s.d / V;
  // Long inputs: as many tokens as make one piece per thread, whose cosines then serve every head of both
  // tensors. Short ones: fewer tokens and several threads to a piece's heads, so that two blocks come to
  // each SM; when tokens alone are too few for that, the heads are split over blocks too.
  const long long spread = std::max<long long>(1, rows / (2LL * sm_count()));
  p.tt = static_cast<int>(std::min<long long>(spread, std::max(1, kta::ROPE_THREADS / p.n_items)));
  p.lanes = std::max(1, kta::ROPE_THREADS / (p.tt * p.n_items));
  const int Hall = Hs[0] + Hs[1];
  const long long gx = (rows + p.tt - 1) / p.tt;
  if ((r = check_grid(gx))) return r;
  const long long want = std::max<long long>(1, 2LL * sm_count() / gx);
  const int step = static_cast<int>(std::min<long long>(Hall, std::max<long long>(p.lanes, (Hall + want - 1) / want)));
  p.head_step = step;
  const long long gy = (Hall + step - 1) / step;
  if (gy > 65535) return fail(KTA_ERR_UNSUPPORTED, "too many heads");
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  cudaStream_t st = as_stream(stream);
  return s.dtype == KTA_BF16 ? launch_rope<__nv_bfloat16>(p, W, grid, st) : launch_rope<float>(p, W, grid, st);
}

// Tokens are counted in 32 bits; a run or segment, and the rows fetched ahead, may end behind the last one.
kta_status check_rows(int B, int L) {
  if (static_cast<long long>(B) * L >= (1LL << 31) - (1 << 16))
    return fail(KTA_ERR_UNSUPPORTED, "B*L must be < 2^31 - 2^16");
  return KTA_OK;
}

// ------------------------------------------------------------------------- short convolution

kta_status check_conv(const kta_short_conv* c) {
  kta_status r;
  if (!c) return fail(KTA_ERR_INVALID_ARG, "null convolution description");
  if (c->B < 1 || c->L < 1 || c->D < 1) return fail(KTA_ERR_INVALID_ARG, "B, L, D must be >= 1");
  if (c->dtype != KTA_BF16 && c->dtype != KTA_F32) return fail(KTA_ERR_INVALID_ARG, "bad dtype");
  if (c->K < 2 || c->K > 4) return fail(KTA_ERR_UNSUPPORTED, "K must be 2, 3 or 4 (got %d)", c->K);
  if (c->D % 8) return fail(KTA_ERR_ALIGNMENT, "D must be a multiple of 8 (16-byte rows)");
  if ((r = check_rows(c->B, c->L))) return r;
  if (c->D >= (1 << 28)) return fail(KTA_ERR_UNSUPPORTED, "D must be < 2^28");
  if (reinterpret_cast<uintptr_t>(c->lens) & 3) return fail(KTA_ERR_ALIGNMENT, "lens must be 4-byte aligned");
  return KTA_OK;
}

// Tokens per run: long runs re-read fewer rows of their neighbours, short ones fill the card (768 threads
// on each SM).
int conv_run(const kta_short_conv* c) {
  int run = kta::SC_RUN;
  while (run > kta::SC_MIN_RUN && static_cast<long long>(c->B) * ((c->L + run - 1) / run) * (c->D / kta::SC_V) <
                                      768LL * sm_count())
    run /= 2;
  return run;
}

// Backward: runs are stretched towards a whole number of turns of the card where that shortens the path of its
// busiest SM. There a row of k blocks takes 2 + 4 k units: one for each warp, and two whatever their number.
// (Fits 120 measured plans to 2 %; one choice in 60 was the slower by more than that: 4 %.) us with runs of
// 64 / of the stretched length, and the turns of the card that the stretched blocks fill:
//   stretched: 2 x 3,600 x 4,096  67.0 / 58.3 (0.97), 2 x 12,000 x 2,048  97.1 / 91.0 (2.00),
//     8 x 1,759 x 7,936  197.5 / 187.7 (4.19);
//   kept: 8 x 768 x 5,120  66.6 / 80.8 (0.54), 24 x 512 x 4,096  97.2 / 103.3 (1.30),
//     8 x 4,096 x 2,048  119.9 / 126.0 (2.81).
int conv_bwd_run(const kta_short_conv* c) {
  const int run = conv_run(c);
  const long long per = static_cast<long long>(c->B) * ((c->D / kta::SC_V + kta::SC_BWD_X - 1) / kta::SC_BWD_X);
  const long long sms = sm_count(), slots = kta::SC_BWD_BLOCKS * sms;
  auto blocks = [&](int r) {                               // of the grid, as the launch counts them
    return per * (((c->L + r - 1) / r + kta::SC_BWD_Y - 1) / kta::SC_BWD_Y);
  };
  auto path = [&](int r) {
    const long long n = blocks(r), rest = (n % slots + sms - 1) / sms;
    return (r + c->K - 1) * (n / slots * (2 + 4 * kta::SC_BWD_BLOCKS) + (rest ? 2 + 4 * rest : 0));
  };
  const long long fit = blocks(run) / slots * slots / per;       // blocks of runs per sequence
  if (run < kta::SC_RUN || fit < 1) return run;
  const int longer = static_cast<int>((c->L + fit * kta::SC_BWD_Y - 1) / (fit * kta::SC_BWD_Y));
  return longer > run && path(longer) < path(run) ? longer : run;
}

kta::ConvParams conv_params(const kta_short_conv* c, bool bwd) {
  kta::ConvParams p{};
  p.x = c->x;
  p.S0 = c->S0;
  p.w = c->w;
  p.bias = c->bias;
  p.lens = c->lens;
  p.B = c->B;
  p.L = c->L;
  p.D = c->D;
  p.silu = c->silu;
  p.run = bwd ? conv_bwd_run(c) : conv_run(c);
  p.runs = (c->L + p.run - 1) / p.run;
  p.nch = c->D / kta::SC_V;
  return p;
}

long long conv_bwd_blocks(const kta::ConvParams& p) {   // (sequence, block of runs)
  return static_cast<long long>(p.B) * ((p.runs + kta::SC_BWD_Y - 1) / kta::SC_BWD_Y);
}

template <typename T, int K>
kta_status launch_conv_fwd(const kta::ConvParams& p, long long blocks, cudaStream_t st) {
  TraceScope ts("short_conv_fwd", st);
  const auto kern = p.silu ? kta::short_conv_fwd_kernel<T, K, true> : kta::short_conv_fwd_kernel<T, K, false>;
  kern<<<static_cast<unsigned>(blocks), kta::SC_THREADS, 0, st>>>(p);
  KTA_CUDA(cudaGetLastError());
  return KTA_OK;
}

template <typename T, int K>
kta_status launch_conv_bwd(const kta::ConvParams& p, long long blocks, long long rows, float* dw,
                           float* dbias, cudaStream_t st) {
  {
    TraceScope ts("short_conv_bwd", st);
    const auto kern = p.silu ? kta::short_conv_bwd_kernel<T, K, true> : kta::short_conv_bwd_kernel<T, K, false>;
    kern<<<static_cast<unsigned>(blocks), kta::SC_BWD_X * kta::SC_BWD_Y, 0, st>>>(p);
    KTA_CUDA(cudaGetLastError());
  }
  TraceScope ts("short_conv_dw", st);
  const unsigned g = static_cast<unsigned>(((K + 1) * static_cast<long long>(p.D) + 31) / 32);
  KTA_CUDA(launch_next(kta::short_conv_dw_kernel<K>, g, 256, 0, st, p.part, rows, p.D, dw, dbias));
  return KTA_OK;
}

kta_status conv_fwd_common(const kta_short_conv* c, void* o, void* S_out, void* stream) {
  kta_status r;
  if ((r = check_conv(c))) return r;
  const size_t es = elem_size(c->dtype);
  const size_t n = static_cast<size_t>(c->B) * c->L * c->D * es;
  const size_t ns = static_cast<size_t>(c->B) * (c->K - 1) * c->D * es;
  const size_t nw = static_cast<size_t>(c->D) * c->K * 4;
  const bool in_place = S_out && S_out == c->S0;
  const Span v[] = {{c->x, n, false, true, "x"},
                    {c->w, nw, false, true, "w"},
                    {c->bias, static_cast<size_t>(c->D) * 4, false, false, "bias"},
                    {in_place ? nullptr : c->S0, ns, false, false, "S0"},
                    {c->lens, static_cast<size_t>(c->B) * 4, false, false, "lens", 4},
                    {o, n, true, true, "o"},
                    {S_out, ns, true, false, "S_out"}};
  if ((r = check_spans(v, 7))) return r;
  kta::ConvParams p = conv_params(c, false);
  p.o = o;
  p.S_out = S_out;
  const long long blocks =
      (static_cast<long long>(p.B) * p.runs * p.nch + kta::SC_THREADS - 1) / kta::SC_THREADS;
  if ((r = check_grid(blocks))) return r;
  cudaStream_t st = as_stream(stream);
  if (c->dtype == KTA_BF16) {
    if (c->K == 4) return launch_conv_fwd<__nv_bfloat16, 4>(p, blocks, st);
    if (c->K == 3) return launch_conv_fwd<__nv_bfloat16, 3>(p, blocks, st);
    return launch_conv_fwd<__nv_bfloat16, 2>(p, blocks, st);
  }
  if (c->K == 4) return launch_conv_fwd<float, 4>(p, blocks, st);
  if (c->K == 3) return launch_conv_fwd<float, 3>(p, blocks, st);
  return launch_conv_fwd<float, 2>(p, blocks, st);
}

// ------------------------------------------------------------------------- state-space scan

kta_status check_ssm(const kta_ssm* c) {
  kta_status r;
  if (!c) return fail(KTA_ERR_INVALID_ARG, "null scan description");
  if (c->B < 1 || c->L < 1 || c->D < 1 || c->N < 1 || c->G < 1)
    return fail(KTA_ERR_INVALID_ARG, "B, L, D, N, G must be >= 1");
  if (c->dtype != KTA_BF16 && c->dtype != KTA_F32) return fail(KTA_ERR_INVALID_ARG, "bad dtype");
  if (c->N > kta::SSM_MAX_N)
    return fail(KTA_ERR_UNSUPPORTED, "N must be <= %d (got %d)", kta::SSM_MAX_N, c->N);
  if (c->D % c->G) return fail(KTA_ERR_INVALID_ARG, "G must divide D");
  if (c->D / c->G % 8)
    return fail(KTA_ERR_ALIGNMENT, "the channels of a group must be a multiple of 8 (16-byte rows)");
  if ((r = check_rows(c->B, c->L))) return r;
  if (c->D >= (1 << 26)) return fail(KTA_ERR_UNSUPPORTED, "D must be < 2^26");
  if (reinterpret_cast<uintptr_t>(c->lens) & 3) return fail(KTA_ERR_ALIGNMENT, "lens must be 4-byte aligned");
  return KTA_OK;
}

constexpr int kSsmInputs = 10;

void ssm_inputs(const kta_ssm* c, Span* v) {
  const size_t es = elem_size(c->dtype), rows = static_cast<size_t>(c->B) * c->L;
  const size_t n = rows * c->D * es, bc = rows * c->G * c->N * es, d4 = static_cast<size_t>(c->D) * 4;
  v[0] = {c->u, n, false, true, "u"};
  v[1] = {c->dt, n, false, true, "dt"};
  v[2] = {c->A, d4 * c->N, false, true, "A"};
  v[3] = {c->Bm, bc, false, true, "B", unsigned(es)};
  v[4] = {c->Cm, bc, false, true, "C", unsigned(es)};
  v[5] = {c->D_skip, d4, false, false, "D_skip"};
  v[6] = {c->z, n, false, false, "z"};
  v[7] = {c->dt_bias, d4, false, false, "dt_bias"};
  v[8] = {c->S0, d4 * c->N * c->B, false, false, "S0"};
  v[9] = {c->lens, static_cast<size_t>(c->B) * 4, false, false, "lens", 4};
}

kta::SsmParams ssm_params(const kta_ssm* c) {
  kta::SsmParams p{};
  p.u = c->u;
  p.dt = c->dt;
  p.Bm = c->Bm;
  p.Cm = c->Cm;
  p.z = c->z;
  p.A = c->A;
  p.Dskip = c->D_skip;
  p.dt_bias = c->dt_bias;
  p.S0 = c->S0;
  p.lens = c->lens;
  p.B = c->B;
  p.L = c->L;
  p.D = c->D;
  p.N = c->N;
  p.G = c->G;
  p.Dg = c->D / c->G;
  p.cbg = (p.Dg + kta::SSM_CH - 1) / kta::SSM_CH;
  const uintptr_t bc = static_cast<uintptr_t>(c->N) * elem_size(c->dtype) |
                       reinterpret_cast<uintptr_t>(c->Bm) | reinterpret_cast<uintptr_t>(c->Cm);
  p.bc_bytes = bc % 16 == 0 ? 16 : bc % 8 == 0 ? 8 : bc % 4 == 0 ? 4 : 0;
  return p;
}

// States per lane: the smallest power of two that holds N in four lanes.
int ssm_ns(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }

// States a lane of the forward pass holds: the power of two, at least 4, that holds N.
int ssm_np(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : 32; }

// Segments of the forward pass. Every exponential of a segment but the last is computed twice (end
// state, then outputs), so a sequence stays whole once its warps give each of the SM's four
// schedulers one (B 8, D 4,096, N 16: 551 us whole, 660 in two); with fewer, segments fill the four
// warps that fit on each (B 4, L 2,048, D 2,048: 475 us whole, 202 in nine). A segment shorter
// than 32 tokens costs as much to start as it gains (B 1, L 512, D 1,024: 37 us at 64, 26 at 32, 24 at 16).
void ssm_plan(kta::SsmParams& p) {
  const long long warps = static_cast<long long>(p.B) * p.G * p.cbg;
  const long long one = 4LL * sm_count(), full = one * (ssm_np(p.N) > 16 ? 3 : 4);
  long long n = warps >= one ? 1 : std::max<long long>(1, std::min<long long>(full / warps, p.L / 32));
  p.seg = static_cast<int>((p.L + n - 1) / n);
  p.seg = (p.seg + kta::SSM_TT - 1) / kta::SSM_TT * kta::SSM_TT;
  p.nseg = (p.L + p.seg - 1) / p.seg;
}

size_t ssm_fwd_states_bytes(const kta::SsmParams& p) {
  return mixer_round(static_cast<size_t>(p.B) * p.nseg * p.D * ssm_np(p.N) * 4);
}

size_t ssm_fwd_bytes(const kta::SsmParams& p) {
  return p.nseg == 1 ? 0 : ssm_fwd_states_bytes(p) + mixer_round(static_cast<size_t>(p.B) * p.nseg * p.D * 4);
}

template <typename T, int NP>
kta_status launch_ssm_fwd(const kta::SsmParams& p, cudaStream_t st) {
  constexpr int W = kta::SSM_THREADS / 32;
  const long long per = static_cast<long long>(p.B) * p.G * p.cbg;
  const long long states = static_cast<long long>(p.B) * p.D * NP;
  const size_t smem_out = W * sizeof(kta::SsmFwdSmem<T, NP, true>);
  const size_t smem_loc = W * sizeof(kta::SsmFwdSmem<T, NP, false>);
  kta_status r;
  if ((r = check_grid((per * p.nseg + W - 1) / W)) || (r = check_grid((states + 255) / 256)) ||
      (r = set_smem_attr(kta::ssm_fwd_kernel<T, NP, true>, smem_out)))
    return r;
  if (p.nseg > 1) {
    if ((r = set_smem_attr(kta::ssm_fwd_kernel<T, NP, false>, smem_loc))) return r;
    {
      TraceScope ts("ssm_local", st);
      kta::ssm_fwd_kernel<T, NP, false>
          <<<static_cast<unsigned>((per * (p.nseg - 1) + W - 1) / W), kta::SSM_THREADS, smem_loc, st>>>(p);
      KTA_CUDA(cudaGetLastError());
    }
    TraceScope ts("ssm_carry", st);
    kta::ssm_fwd_carry_kernel<<<static_cast<unsigned>((states + 255) / 256), 256, 0, st>>>(p, NP);
    KTA_CUDA(cudaGetLastError());
  }
  TraceScope ts("ssm_fwd", st);
  kta::ssm_fwd_kernel<T, NP, true>
      <<<static_cast<unsigned>((per * p.nseg + W - 1) / W), kta::SSM_THREADS, smem_out, st>>>(p);
  KTA_CUDA(cudaGetLastError());
  return KTA_OK;
}

template <typename T, int NS>
kta_status launch_ssm_step(const kta::SsmParams& p, cudaStream_t st) {
  const int gy = (p.B + kta::SSM_STEP_B - 1) / kta::SSM_STEP_B;
  if (gy > 65535) return fail(KTA_ERR_UNSUPPORTED, "a step takes at most %d sequences", 65535 * kta::SSM_STEP_B);
  const dim3 grid((static_cast<unsigned>(p.D) * 4 + kta::SSM_THREADS - 1) / kta::SSM_THREADS, static_cast<unsigned>(gy));
  TraceScope ts("ssm_step", st);
  kta::ssm_step_kernel<T, NS><<<grid, kta::SSM_THREADS, 0, st>>>(p);
  KTA_CUDA(cudaGetLastError());
  return KTA_OK;
}

void ssm_bwd_plan(kta::SsmBwdParams& p) {
  p.f.seg = kta::SSM_BWD_SEG;
  p.f.nseg = (p.f.L + p.f.seg - 1) / p.f.seg;
  const int np = ssm_np(p.f.N);
  const int ch = np == 4   ? kta::SsmBwdCfg<4>::BCH
                 : np == 8 ? kta::SsmBwdCfg<8>::BCH
                 : np == 16 ? kta::SsmBwdCfg<16>::BCH
                            : kta::SsmBwdCfg<32>::BCH;
  p.cbg = (p.f.Dg + ch - 1) / ch;
}

struct SsmBwdWs {
  size_t h, g, d, c, bc, total;
};

SsmBwdWs ssm_bwd_ws(const kta::SsmBwdParams& p) {
  const size_t segs = static_cast<size_t>(p.f.B) * p.f.nseg * p.f.D;
  SsmBwdWs w;
  size_t at = 0;
  auto put = [&](size_t n) {
    const size_t o = at;
    at += mixer_round(n * 4);
    return o;
  };
  w.h = put(segs * ssm_np(p.f.N));
  w.g = put(segs * ssm_np(p.f.N));
  w.d = put(segs);
  w.c = put(segs * 2);
  w.bc = put(static_cast<size_t>(p.f.G) * p.cbg * p.f.B * p.f.L * 2 * p.f.N);
  w.total = at;
  return w;
}

template <typename T, int NP>
kta_status launch_ssm_bwd(const kta::SsmBwdParams& p, cudaStream_t st) {
  constexpr int W = kta::SSM_THREADS / 32;
  const long long segs = static_cast<long long>(p.f.B) * p.f.nseg * p.f.G;
  const long long blocks_l = (segs * p.f.cbg + W - 1) / W, blocks_m = segs * p.cbg;
  const long long states = static_cast<long long>(p.f.B) * p.f.D * NP;
  const long long bc = static_cast<long long>(p.f.B) * p.f.L * p.f.G * 2 * p.f.N;
  const long long bc_blocks = (bc + 255) / 256;
  const long long param_blocks = (static_cast<long long>(p.f.D) * p.f.N + 31) / 32 + (2LL * p.f.D + 31) / 32;
  kta_status r;
  if ((r = check_grid(blocks_l)) || (r = check_grid(blocks_m)) || (r = check_grid((states + 255) / 256)) ||
      (r = check_grid(bc_blocks + param_blocks)))
    return r;
  const size_t smem_l = W * sizeof(kta::SsmLocalSmem<T, NP>), smem_m = sizeof(kta::SsmMainSmem<T, NP>);
  if ((r = set_smem_attr(kta::ssm_bwd_local_kernel<T, NP>, smem_l)) ||
      (r = set_smem_attr(kta::ssm_bwd_main_kernel<T, NP>, smem_m)))
    return r;
  {
    TraceScope ts("ssm_bwd_local", st);
    kta::ssm_bwd_local_kernel<T, NP><<<static_cast<unsigned>(blocks_l), kta::SSM_THREADS, smem_l, st>>>(p);
    KTA_CUDA(cudaGetLastError());
  }
  {
    TraceScope ts("ssm_bwd_carry", st);
    KTA_CUDA(launch_next(kta::ssm_bwd_carry_kernel, dim3(static_cast<unsigned>((states + 255) / 256), 2), 256, 0, st,
                         p, NP));
  }
  {
    TraceScope ts("ssm_bwd_main", st);
    KTA_CUDA(launch_next(kta::ssm_bwd_main_kernel<T, NP>, static_cast<unsigned>(blocks_m), kta::SSM_THREADS, smem_m,
                         st, p));
  }
  TraceScope ts("ssm_bwd_sums", st);
  KTA_CUDA(launch_next(kta::ssm_bwd_sums_kernel<T>, static_cast<unsigned>(bc_blocks + param_blocks), 256, 0, st, p,
                       NP, static_cast<unsigned>(bc_blocks)));
  return KTA_OK;
}

#define KTA_SSM_FWD_DISPATCH(fn, dtype, N, ...)                                 \
  do {                                                                          \
    const int np_ = ssm_np(N);                                                  \
    if ((dtype) == KTA_BF16) {                                                  \
      if (np_ == 4) return fn<__nv_bfloat16, 4>(__VA_ARGS__);                   \
      if (np_ == 8) return fn<__nv_bfloat16, 8>(__VA_ARGS__);                   \
      if (np_ == 16) return fn<__nv_bfloat16, 16>(__VA_ARGS__);                 \
      return fn<__nv_bfloat16, 32>(__VA_ARGS__);                                \
    }                                                                           \
    if (np_ == 4) return fn<float, 4>(__VA_ARGS__);                             \
    if (np_ == 8) return fn<float, 8>(__VA_ARGS__);                             \
    if (np_ == 16) return fn<float, 16>(__VA_ARGS__);                           \
    return fn<float, 32>(__VA_ARGS__);                                          \
  } while (0)

#define KTA_SSM_DISPATCH(fn, dtype, N, ...)                                     \
  do {                                                                          \
    const int ns_ = ssm_ns(N);                                                  \
    if ((dtype) == KTA_BF16) {                                                  \
      if (ns_ == 1) return fn<__nv_bfloat16, 1>(__VA_ARGS__);                   \
      if (ns_ == 2) return fn<__nv_bfloat16, 2>(__VA_ARGS__);                   \
      if (ns_ == 4) return fn<__nv_bfloat16, 4>(__VA_ARGS__);                   \
      return fn<__nv_bfloat16, 8>(__VA_ARGS__);                                 \
    }                                                                           \
    if (ns_ == 1) return fn<float, 1>(__VA_ARGS__);                             \
    if (ns_ == 2) return fn<float, 2>(__VA_ARGS__);                             \
    if (ns_ == 4) return fn<float, 4>(__VA_ARGS__);                             \
    return fn<float, 8>(__VA_ARGS__);                                           \
  } while (0)

kta_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return KTA_OK;
  if (!ws || have < need)
    return fail(KTA_ERR_INVALID_ARG, "the workspace has %zu bytes; this call needs %zu", ws ? have : 0, need);
  if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(KTA_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  return KTA_OK;
}

}  // namespace

extern "C" {

kta_status kta_rope_freqs(int dims, double base, int scaling, double factor, double orig_len,
                          double beta_fast, double beta_slow, double* freqs, float* mscale) {
  if (!freqs || !mscale) return fail(KTA_ERR_INVALID_ARG, "null output");
  if (dims < 2 || dims % 2 || dims > 2 * kta::ROPE_MAX_PAIRS)
    return fail(KTA_ERR_INVALID_ARG, "dims must be even and in [2, %d]", 2 * kta::ROPE_MAX_PAIRS);
  if (!(base > 0) || !std::isfinite(base)) return fail(KTA_ERR_INVALID_ARG, "base must be > 0");
  if (scaling < KTA_ROPE_PLAIN || scaling > KTA_ROPE_BY_PARTS) return fail(KTA_ERR_INVALID_ARG, "bad scaling");
  if (scaling != KTA_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor)))
    return fail(KTA_ERR_INVALID_ARG, "factor must be >= 1");
  if (scaling == KTA_ROPE_BY_PARTS &&
      (!(orig_len > 0) || !std::isfinite(orig_len) || !(beta_slow >= 0) || !(beta_fast > beta_slow) ||
       !std::isfinite(beta_fast)))
    return fail(KTA_ERR_INVALID_ARG, "need orig_len > 0 and beta_fast > beta_slow >= 0");
  *mscale = 1.f;
  if (scaling == KTA_ROPE_BASE && dims > 2) base *= std::pow(factor, dims / (dims - 2.0));
  for (int i = 0; i < dims / 2; ++i) {
    double f = std::pow(base, -2.0 * i / dims);
    if (scaling == KTA_ROPE_LINEAR || (scaling == KTA_ROPE_BASE && dims == 2)) f /= factor;
    if (scaling == KTA_ROPE_BY_PARTS) {
      const double turns = orig_len * f / 6.283185307179586477;
      const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = f;
  }
  if (scaling == KTA_ROPE_BY_PARTS) *mscale = static_cast<float>(0.1 * std::log(factor) + 1.0);
  return KTA_OK;
}

kta_status kta_rope_fwd(const kta_rope* cfg, const void* x, void* o, const void* x2, void* o2,
                        kta_shape s, int H, int ld_heads, int H2, int ld_heads2, void* stream) {
  return rope_common(cfg, x, o, x2, o2, s, H, ld_heads, H2, ld_heads2, 1.f, stream);
}

kta_status kta_rope_bwd(const kta_rope* cfg, const void* dout, void* dx, const void* dout2, void* dx2,
                        kta_shape s, int H, int ld_heads, int H2, int ld_heads2, void* stream) {
  return rope_common(cfg, dout, dx, dout2, dx2, s, H, ld_heads, H2, ld_heads2, -1.f, stream);
}

kta_status kta_short_conv_fwd(const kta_short_conv* c, void* o, void* S_out, void* stream) {
  return conv_fwd_common(c, o, S_out, stream);
}

size_t kta_short_conv_bwd_workspace(const kta_short_conv* c) {
  if (check_conv(c)) return 0;
  return mixer_round(static_cast<size_t>(conv_bwd_blocks(conv_params(c, true))) * (c->K + 1) * c->D * 4);
}

kta_status kta_short_conv_bwd(const kta_short_conv* c, const void* dout, const void* dS_out, void* dx,
                              float* dw, float* dbias, void* dS0, void* ws, size_t ws_bytes,
                              void* stream) {
  kta_status r;
  if ((r = check_conv(c))) return r;
  if (dS0 && !c->S0) return fail(KTA_ERR_INVALID_ARG, "dS0 without S0");
  const size_t es = elem_size(c->dtype);
  const size_t n = static_cast<size_t>(c->B) * c->L * c->D * es;
  const size_t ns = static_cast<size_t>(c->B) * (c->K - 1) * c->D * es;
  const size_t nw = static_cast<size_t>(c->D) * c->K * 4, nb = static_cast<size_t>(c->D) * 4;
  const size_t need = kta_short_conv_bwd_workspace(c);
  if ((r = check_ws(ws, ws_bytes, need))) return r;
  const Span v[] = {{c->x, n, false, true, "x"},       {c->w, nw, false, true, "w"},
                    {c->bias, nb, false, false, "bias"}, {c->S0, ns, false, false, "S0"},
                    {dout, n, false, true, "dout"},    {dS_out, ns, false, false, "dS_out"},
                    {dx, n, true, true, "dx"},         {dw, nw, true, true, "dw"},
                    {dbias, nb, true, false, "dbias"}, {dS0, ns, true, false, "dS0"},
                    {c->lens, static_cast<size_t>(c->B) * 4, false, false, "lens", 4},
                    {ws, need, true, false, "the workspace"}};
  if ((r = check_spans(v, 12))) return r;
  kta::ConvParams p = conv_params(c, true);
  p.dout = dout;
  p.dS_out = dS_out;
  p.dx = dx;
  p.dS0 = dS0;
  p.part = static_cast<float*>(ws);
  const long long rows = conv_bwd_blocks(p);
  const long long blocks = rows * ((p.nch + kta::SC_BWD_X - 1) / kta::SC_BWD_X);
  if ((r = check_grid(blocks))) return r;
  cudaStream_t st = as_stream(stream);
  if (c->dtype == KTA_BF16) {
    if (c->K == 4) return launch_conv_bwd<__nv_bfloat16, 4>(p, blocks, rows, dw, dbias, st);
    if (c->K == 3) return launch_conv_bwd<__nv_bfloat16, 3>(p, blocks, rows, dw, dbias, st);
    return launch_conv_bwd<__nv_bfloat16, 2>(p, blocks, rows, dw, dbias, st);
  }
  if (c->K == 4) return launch_conv_bwd<float, 4>(p, blocks, rows, dw, dbias, st);
  if (c->K == 3) return launch_conv_bwd<float, 3>(p, blocks, rows, dw, dbias, st);
  return launch_conv_bwd<float, 2>(p, blocks, rows, dw, dbias, st);
}

size_t kta_ssm_scan_fwd_workspace(const kta_ssm* c) {
  if (check_ssm(c)) return 0;
  kta::SsmParams p = ssm_params(c);
  ssm_plan(p);
  return ssm_fwd_bytes(p);
}

kta_status kta_ssm_scan_fwd(const kta_ssm* c, void* y, float* S_out, void* ws, size_t ws_bytes,
                            void* stream) {
  kta_status r;
  if ((r = check_ssm(c))) return r;
  kta::SsmParams p = ssm_params(c);
  ssm_plan(p);
  const size_t need = ssm_fwd_bytes(p);
  if ((r = check_ws(ws, ws_bytes, need))) return r;
  Span v[kSsmInputs + 3];
  ssm_inputs(c, v);
  v[kSsmInputs] = {y, v[0].bytes, true, true, "y"};
  v[kSsmInputs + 1] = {S_out, v[8].bytes, true, false, "S_out"};
  v[kSsmInputs + 2] = {need ? ws : nullptr, need, true, false, "the workspace"};
  if ((r = check_spans(v, kSsmInputs + 3))) return r;
  p.y = y;
  p.S_out = S_out;
  if (need) {
    p.seg_h = static_cast<float*>(ws);
    p.seg_d = reinterpret_cast<float*>(static_cast<char*>(ws) + ssm_fwd_states_bytes(p));
  }
  cudaStream_t st = as_stream(stream);
  KTA_SSM_FWD_DISPATCH(launch_ssm_fwd, c->dtype, c->N, p, st);
}

kta_status kta_ssm_scan_step(const kta_ssm* c, void* y, float* S_out, void* stream) {
  kta_status r;
  if ((r = check_ssm(c))) return r;
  if (c->L != 1) return fail(KTA_ERR_INVALID_ARG, "a step takes one token (L = %d)", c->L);
  if (c->lens) return fail(KTA_ERR_INVALID_ARG, "a step takes no lengths");
  if (!c->S0) return fail(KTA_ERR_INVALID_ARG, "S0 must not be null");
  Span v[kSsmInputs + 2];
  ssm_inputs(c, v);
  v[kSsmInputs] = {y, v[0].bytes, true, true, "y"};
  v[kSsmInputs + 1] = {S_out, v[8].bytes, true, true, "S_out"};
  if (S_out == c->S0) v[8].p = nullptr;   // in place: each state is read and written by one thread
  if ((r = check_spans(v, kSsmInputs + 2))) return r;
  kta::SsmParams p = ssm_params(c);
  p.nseg = 1;
  p.y = y;
  p.S_out = S_out;
  cudaStream_t st = as_stream(stream);
  KTA_SSM_DISPATCH(launch_ssm_step, c->dtype, c->N, p, st);
}

size_t kta_ssm_scan_bwd_workspace(const kta_ssm* c) {
  if (check_ssm(c)) return 0;
  kta::SsmBwdParams p{};
  p.f = ssm_params(c);
  ssm_bwd_plan(p);
  return ssm_bwd_ws(p).total;
}

kta_status kta_ssm_scan_bwd(const kta_ssm* c, const kta_ssm_grads* g, void* ws, size_t ws_bytes,
                            void* stream) {
  kta_status r;
  if ((r = check_ssm(c))) return r;
  if (!g) return fail(KTA_ERR_INVALID_ARG, "null gradient description");
  if ((g->dz != nullptr) != (c->z != nullptr)) return fail(KTA_ERR_INVALID_ARG, "dz goes with z");
  if (g->dD_skip && !c->D_skip) return fail(KTA_ERR_INVALID_ARG, "dD_skip without D_skip");
  kta::SsmBwdParams p{};
  p.f = ssm_params(c);
  ssm_bwd_plan(p);
  const SsmBwdWs w = ssm_bwd_ws(p);
  if ((r = check_ws(ws, ws_bytes, w.total))) return r;
  Span v[kSsmInputs + 12];
  ssm_inputs(c, v);
  const size_t n = v[0].bytes, bc = v[3].bytes, d4 = static_cast<size_t>(c->D) * 4, sb = v[8].bytes;
  int k = kSsmInputs;
  v[k++] = {g->dout, n, false, true, "dout"};
  v[k++] = {g->dS_out, sb, false, false, "dS_out"};
  v[k++] = {g->du, n, true, true, "du"};
  v[k++] = {g->ddt, n, true, true, "ddt"};
  v[k++] = {g->dA, d4 * c->N, true, true, "dA"};
  v[k++] = {g->dB, bc, true, true, "dB", v[3].align};
  v[k++] = {g->dC, bc, true, true, "dC", v[3].align};
  v[k++] = {g->dD_skip, d4, true, false, "dD_skip"};
  v[k++] = {g->dz, n, true, false, "dz"};
  v[k++] = {g->ddt_bias, d4, true, false, "ddt_bias"};
  v[k++] = {g->dS0, sb, true, false, "dS0"};
  v[k++] = {ws, w.total, true, true, "the workspace"};
  if ((r = check_spans(v, k))) return r;
  p.dout = g->dout;
  p.dS_out = g->dS_out;
  p.du = g->du;
  p.ddt = g->ddt;
  p.dz = g->dz;
  p.dB = g->dB;
  p.dC = g->dC;
  p.dA = g->dA;
  p.dD = g->dD_skip;
  p.ddt_bias = g->ddt_bias;
  p.dS0 = g->dS0;
  char* base = static_cast<char*>(ws);
  p.f.seg_h = reinterpret_cast<float*>(base + w.h);
  p.seg_g = reinterpret_cast<float*>(base + w.g);
  p.f.seg_d = reinterpret_cast<float*>(base + w.d);
  p.part_c = reinterpret_cast<float*>(base + w.c);
  p.part_bc = reinterpret_cast<float*>(base + w.bc);
  cudaStream_t st = as_stream(stream);
  KTA_SSM_FWD_DISPATCH(launch_ssm_bwd, c->dtype, c->N, p, st);
}

}  // extern "C"
