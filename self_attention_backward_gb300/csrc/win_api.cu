// win_api.cu -- C entry points of the sliding-window attention family: argument
// checks and dispatch (contracts in include/psa_attn.h).  Every argument is
// checked before anything is launched.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "psa_attn.h"
#include "psa_internal.h"
#include "win_internal.h"

namespace {

using psa::View;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return psa::set_last_error(code, buf);
}
int done(int rc, const std::string& err) { return rc ? fail(rc, "%s", err.c_str()) : psa::set_last_error(PSA_OK, ""); }
int ok() { return psa::set_last_error(PSA_OK, ""); }

constexpr long long kMaxElems = 1ll << 40;       // as for psa_attn_*: indexes stay far below 2^62
constexpr int kMaxRows = 1 << 30;                // rows, keys, slots: sums of two stay in 32 bits

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool dtype_ok(int t) { return t == PSA_F32 || t == PSA_BF16; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// A view of a [B, heads, N, d] tensor that is not empty.  An output's elements
// must be distinct: no zero stride along a dimension longer than 1.
int check_view(const char* name, const psa_attn_view* v, long long B, long long heads, long long N, int d, bool out,
               View* to) {
    if (!v) return fail(PSA_ERR_ARG, "%s view is NULL", name);
    *to = View{v->base, v->batch_stride, v->head_stride, v->pos_stride, v->feat_stride};
    if (B == 0 || heads == 0 || N == 0) return PSA_OK;
    if (!v->base) return fail(PSA_ERR_ARG, "%s view's base is NULL", name);
    if (!aligned(v->base, 16)) return fail(PSA_ERR_ALIGN, "%s view's base is not 16-byte aligned", name);
    const long long n[4] = {B, heads, N, d}, s[4] = {to->sB, to->sH, to->sN, to->sJ};
    long long reach = 0;
    for (int i = 0; i < 4; ++i) {
        if (s[i] < 0) return fail(PSA_ERR_ARG, "%s view has a negative stride", name);
        if (out && s[i] == 0 && n[i] > 1) return fail(PSA_ERR_ARG, "%s view has a zero stride: its elements coincide", name);
        if (n[i] > 1) {
            if (s[i] > kMaxElems || (n[i] - 1) * s[i] > kMaxElems)
                return fail(PSA_ERR_UNSUPPORTED, "%s view spans more than 2^40 elements", name);
            reach += (n[i] - 1) * s[i];
        }
    }
    if (reach > kMaxElems) return fail(PSA_ERR_UNSUPPORTED, "%s view spans more than 2^40 elements", name);
    return PSA_OK;
}

int check_ptr(const char* name, const void* p, size_t align, int align_code = PSA_ERR_ALIGN) {
    if (!p) return fail(PSA_ERR_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return fail(align_code, "%s is not %zu-byte aligned", name, align);
    return PSA_OK;
}
int check_lens(const char* name, const int* p) {
    return p && !aligned(p, 4) ? fail(PSA_ERR_ALIGN, "%s is not 4-byte aligned", name) : PSA_OK;
}

int check_shape(const psa_win_shape* s, psa::win::Args* a) {
    if (!s) return fail(PSA_ERR_ARG, "shape is NULL");
    if (!dtype_ok(s->dtype)) return fail(PSA_ERR_ARG, "dtype %d is not PSA_F32 or PSA_BF16", s->dtype);
    if (s->B < 0 || s->q_heads < 0 || s->kv_heads < 0 || s->Nq < 0 || s->Nk < 0)
        return fail(PSA_ERR_ARG, "negative size (B=%d q_heads=%d kv_heads=%d Nq=%d Nk=%d)", s->B, s->q_heads, s->kv_heads,
                    s->Nq, s->Nk);
    if (s->window < 1) return fail(PSA_ERR_ARG, "window %d < 1", s->window);
    if (s->sinks < 0) return fail(PSA_ERR_ARG, "sinks %d < 0", s->sinks);
    if (!std::isfinite(s->scale)) return fail(PSA_ERR_ARG, "scale is not finite");
    if (!dim_ok(s->head_dim)) return fail(PSA_ERR_UNSUPPORTED, "head_dim %d not in {16, 32, 64, 128}", s->head_dim);
    if ((s->kv_heads == 0) != (s->q_heads == 0) || (s->kv_heads > 0 && s->q_heads % s->kv_heads))
        return fail(PSA_ERR_ARG, "q_heads %d is not a multiple of kv_heads %d", s->q_heads, s->kv_heads);
    const long long n = std::max(s->Nq, s->Nk);
    if (n > kMaxRows || (double)s->B * s->q_heads * n * s->head_dim > (double)kMaxElems)
        return fail(PSA_ERR_UNSUPPORTED, "problem too large (B=%d q_heads=%d N=%lld d=%d)", s->B, s->q_heads, n, s->head_dim);
    a->B = s->B, a->Hq = s->q_heads, a->Hkv = s->kv_heads, a->Nq = s->Nq, a->Nk = s->Nk, a->d = s->head_dim;
    // a window or sinks past the keys mean the same as Nk of them
    a->window = std::min(s->window, std::max(s->Nk, 1));
    a->sinks = std::min(s->sinks, s->Nk);
    a->scale = s->scale, a->dtype = s->dtype;
    return PSA_OK;
}
bool no_heads(const psa::win::Args& a) { return a.B == 0 || a.Hq == 0; }

// Bytes of the backward's workspace: the row statistics (two fp32 arrays and the
// tensor cores' 16 bytes per row), then the partial sums of the sink rows.
size_t stat_bytes(const psa::win::Args& a) { return (size_t)a.B * a.Hq * psa::win::stat_rows(a.Nq) * 4; }
size_t bwd_workspace(const psa::win::Args& a) {
    if (no_heads(a) || (a.Nq == 0 && a.Nk == 0)) return 0;
    return 6 * stat_bytes(a) + psa::win::part_floats(a, psa::win::far_split(a.Nk, a.window, a.sinks)) * 4;
}

// The layout that TMA and 16-byte stores take: adjacent features, every other
// stride of a dimension longer than 1 a non-zero multiple of 16 bytes.
bool tc_view(const View& v, int B, int heads, int N) {
    auto fits = [](int n, long long s) { return n <= 1 || (s > 0 && s % 8 == 0); };
    return v.sJ == 1 && fits(B, v.sB) && fits(heads, v.sH) && fits(N, v.sN);
}
// The kernels fold the maximum of the raw scores into c = scale log2(e), which
// has to be positive and normal for that.
bool tc_shape(const psa::win::Args& a) { return a.dtype == PSA_BF16 && a.scale >= 1e-30f && a.Nq > 0 && a.Nk > 0; }

// Resolves AUTO; TC is refused where the tensor-core kernels do not take the call.
int pick(int algo, bool tc, bool* use_tc) {
    *use_tc = tc && algo != PSA_ALGO_SIMT;
    if (algo == PSA_ALGO_TC && !tc)
        return fail(PSA_ERR_UNSUPPORTED, "no tensor-core window attention for this dtype, scale or layout");
    return PSA_OK;
}
int check_algo(int algo) {
    if (algo != PSA_ALGO_AUTO && algo != PSA_ALGO_SIMT && algo != PSA_ALGO_TC)
        return fail(PSA_ERR_ARG, "algo %d is not AUTO, SIMT or TC", algo);
    return PSA_OK;
}

int check_cache(const psa_win_cache* c) {
    if (!c) return fail(PSA_ERR_ARG, "cache is NULL");
    if (!dtype_ok(c->dtype)) return fail(PSA_ERR_ARG, "dtype %d is not PSA_F32 or PSA_BF16", c->dtype);
    if (c->B < 0 || c->kv_heads < 0 || c->capacity < 0)
        return fail(PSA_ERR_ARG, "negative size (B=%d kv_heads=%d capacity=%d)", c->B, c->kv_heads, c->capacity);
    if (c->window < 1) return fail(PSA_ERR_ARG, "window %d < 1", c->window);
    if (c->sinks < 0) return fail(PSA_ERR_ARG, "sinks %d < 0", c->sinks);
    if ((long long)c->capacity < (long long)c->sinks + c->window)
        return fail(PSA_ERR_ARG, "capacity %d < sinks %d + window %d", c->capacity, c->sinks, c->window);
    if (!dim_ok(c->head_dim)) return fail(PSA_ERR_UNSUPPORTED, "head_dim %d not in {16, 32, 64, 128}", c->head_dim);
    if (c->capacity > kMaxRows) return fail(PSA_ERR_UNSUPPORTED, "capacity %d > 2^30", c->capacity);
    const psa_attn_view k{c->k, c->batch_stride, c->head_stride, c->slot_stride, 1}, v{c->v, c->batch_stride,
                                                                                      c->head_stride, c->slot_stride, 1};
    View to;
    int rc = check_view("cache k", &k, c->B, c->kv_heads, c->capacity, c->head_dim, true, &to);
    if (!rc) rc = check_view("cache v", &v, c->B, c->kv_heads, c->capacity, c->head_dim, true, &to);
    if (!rc && c->B && c->kv_heads && c->k == c->v) return fail(PSA_ERR_ARG, "cache k and v are the same memory");
    return rc;
}

// A number as the sum of two doubles (some 104 bits); products are split exactly by fma.
struct Two {
    double h, l;
};
Two sum2(double h, double l) {
    const double s = h + l;
    return Two{s, l - (s - h)};                  // |l| is below |h|
}
Two mul2(Two a, Two b) {
    const double p = a.h * b.h;
    return sum2(p, std::fma(a.h, b.h, -p) + (a.h * b.l + a.l * b.h));
}
Two pow2(Two x, int n) {
    Two y{1.0, 0.0};
    for (; n > 0; --n) y = mul2(y, x);
    return y;
}
// theta^(-1/n): one Newton step on theta y^n = 1 from the double result.
Two root(double theta, int n) {
    const Two y{std::pow(theta, -1.0 / n), 0.0}, t = mul2(pow2(y, n), Two{theta, 0.0});
    return sum2(y.h, y.h * ((1.0 - t.h) - t.l) / n);
}
// x / 2 pi in units of 2^-64, rounded (0 <= x <= 1).
unsigned long long turns(Two x) {
    const Two t = mul2(x, Two{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57});
    const double h = std::ldexp(t.h, 64), whole = std::floor(h);
    return (unsigned long long)whole + (unsigned long long)(long long)std::floor((h - whole) + std::ldexp(t.l, 64) + 0.5);
}

int check_plan(const psa_rope_plan* p, int head_dim) {
    if (!p) return fail(PSA_ERR_ARG, "plan is NULL");
    if (!dim_ok(p->head_dim) || p->rot_dim < 2 || p->rot_dim > p->head_dim || p->rot_dim % 2 || p->n_axes < 1 ||
        p->n_axes > 3 || (p->interleaved != 0 && p->interleaved != 1))
        return fail(PSA_ERR_ARG, "plan was not made by psa_rope_plan_init");
    for (int i = 0; i < p->rot_dim / 2; ++i)
        if (p->axis[i] >= p->n_axes) return fail(PSA_ERR_ARG, "plan was not made by psa_rope_plan_init");
    if (head_dim && head_dim != p->head_dim)
        return fail(PSA_ERR_ARG, "plan is for head_dim %d, not %d", p->head_dim, head_dim);
    return PSA_OK;
}
int check_pos(const int* pos, long long axis_stride, long long batch_stride) {
    if (axis_stride < 0 || batch_stride < 0) return fail(PSA_ERR_ARG, "pos has a negative stride");
    return check_ptr("pos", pos, 4);
}

}  // namespace

extern "C" {

int psa_win_attn_fwd(const psa_win_shape* shape, const psa_attn_view* q, const psa_attn_view* k, const psa_attn_view* v,
                     const psa_attn_view* o, float* lse, const int* q_lens, const int* kv_lens, int algo, void* stream) {
    psa::win::Args a{};
    int rc = check_shape(shape, &a);
    if (!rc) rc = check_algo(algo);
    if (rc) return rc;
    if (no_heads(a) || a.Nq == 0) return ok();
    if ((rc = check_view("q", q, a.B, a.Hq, a.Nq, a.d, false, &a.q)) ||
        (rc = check_view("k", k, a.B, a.Hkv, a.Nk, a.d, false, &a.k)) ||
        (rc = check_view("v", v, a.B, a.Hkv, a.Nk, a.d, false, &a.v)) ||
        (rc = check_view("o", o, a.B, a.Hq, a.Nq, a.d, true, &a.o)) || (rc = check_ptr("lse", lse, 16)) ||
        (rc = check_lens("q_lens", q_lens)) || (rc = check_lens("kv_lens", kv_lens)))
        return rc;
    a.lse = lse, a.q_lens = q_lens, a.kv_lens = kv_lens, a.stream = (cudaStream_t)stream;
    bool tc = tc_shape(a) && tc_view(a.q, a.B, a.Hq, a.Nq) && tc_view(a.k, a.B, a.Hkv, a.Nk) &&
              tc_view(a.v, a.B, a.Hkv, a.Nk) && tc_view(a.o, a.B, a.Hq, a.Nq);
    if ((rc = pick(algo, tc, &tc))) return rc;
    std::string err;
    rc = tc ? psa::win::tc_fwd(a, &err) : psa::win::warp_fwd(a, &err);
    return done(rc, err);
}

size_t psa_win_attn_bwd_workspace_bytes(const psa_win_shape* shape) {
    psa::win::Args a{};
    const std::string keep = psa_attn_last_error();
    const int rc = check_shape(shape, &a);
    psa::set_last_error(rc, keep);
    return rc ? 0 : bwd_workspace(a);
}

int psa_win_attn_bwd(const psa_win_shape* shape, const psa_attn_view* q, const psa_attn_view* k, const psa_attn_view* v,
                     const psa_attn_view* o, const float* lse, const psa_attn_view* d_o, const psa_attn_view* dq,
                     const psa_attn_view* dk, const psa_attn_view* dv, const int* q_lens, const int* kv_lens,
                     void* workspace, size_t workspace_bytes, int algo, void* stream) {
    psa::win::Args a{};
    int rc = check_shape(shape, &a);
    if (!rc) rc = check_algo(algo);
    if (rc) return rc;
    if (no_heads(a) || (a.Nq == 0 && a.Nk == 0)) return ok();
    if ((rc = check_view("q", q, a.B, a.Hq, a.Nq, a.d, false, &a.q)) ||
        (rc = check_view("k", k, a.B, a.Hkv, a.Nk, a.d, false, &a.k)) ||
        (rc = check_view("v", v, a.B, a.Hkv, a.Nk, a.d, false, &a.v)) ||
        (rc = check_view("o", o, a.B, a.Hq, a.Nq, a.d, false, &a.o)) ||
        (rc = check_view("d_o", d_o, a.B, a.Hq, a.Nq, a.d, false, &a.dO)) ||
        (rc = check_view("dq", dq, a.B, a.Hq, a.Nq, a.d, true, &a.dq)) ||
        (rc = check_view("dk", dk, a.B, a.Hkv, a.Nk, a.d, true, &a.dk)) ||
        (rc = check_view("dv", dv, a.B, a.Hkv, a.Nk, a.d, true, &a.dv)) ||
        (rc = a.Nq ? check_ptr("lse", lse, 16) : PSA_OK) || (rc = check_lens("q_lens", q_lens)) ||
        (rc = check_lens("kv_lens", kv_lens)))
        return rc;
    const size_t need = bwd_workspace(a);
    if (workspace_bytes < need) return fail(PSA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need) {
        if (!workspace) return fail(PSA_ERR_WORKSPACE, "workspace is NULL");
        if ((rc = check_ptr("workspace", workspace, 16))) return rc;
    }
    a.lse = const_cast<float*>(lse), a.q_lens = q_lens, a.kv_lens = kv_lens, a.stream = (cudaStream_t)stream;
    a.Drow = static_cast<float*>(workspace);
    a.negl = reinterpret_cast<float*>(static_cast<char*>(workspace) + stat_bytes(a));
    a.aug = static_cast<char*>(workspace) + 2 * stat_bytes(a);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 6 * stat_bytes(a));
    bool tc = tc_shape(a) && tc_view(a.q, a.B, a.Hq, a.Nq) && tc_view(a.k, a.B, a.Hkv, a.Nk) &&
              tc_view(a.v, a.B, a.Hkv, a.Nk) && tc_view(a.dO, a.B, a.Hq, a.Nq) && tc_view(a.dq, a.B, a.Hq, a.Nq) &&
              tc_view(a.dk, a.B, a.Hkv, a.Nk) && tc_view(a.dv, a.B, a.Hkv, a.Nk);
    if ((rc = pick(algo, tc, &tc))) return rc;
    std::string err;
    rc = tc ? psa::win::tc_bwd(a, &err) : psa::win::warp_bwd(a, &err);
    return done(rc, err);
}

int psa_rope_plan_init(psa_rope_plan* plan, int head_dim, int rot_dim, int n_axes, const int* sections, double theta,
                       int ladder, int interleaved) {
    if (!plan || !sections) return fail(PSA_ERR_ARG, "plan or sections is NULL");
    if (!dim_ok(head_dim)) return fail(PSA_ERR_UNSUPPORTED, "head_dim %d not in {16, 32, 64, 128}", head_dim);
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
        return fail(PSA_ERR_ARG, "rot_dim %d is not an even number from 2 to head_dim %d", rot_dim, head_dim);
    if (n_axes < 1 || n_axes > 3) return fail(PSA_ERR_ARG, "n_axes %d not in 1..3", n_axes);
    if (!std::isfinite(theta) || theta <= 1.0) return fail(PSA_ERR_ARG, "theta is not a finite number above 1");
    if (ladder != PSA_ROPE_SHARED && ladder != PSA_ROPE_PER_AXIS) return fail(PSA_ERR_ARG, "ladder %d is unknown", ladder);
    const int n = rot_dim / 2;
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0) return fail(PSA_ERR_ARG, "negative section");
        sum += sections[a];
    }
    if (sum != n) return fail(PSA_ERR_ARG, "the sections add up to %lld pairs, not %d", sum, n);
    *plan = psa_rope_plan{};
    plan->head_dim = head_dim, plan->rot_dim = rot_dim, plan->n_axes = n_axes, plan->interleaved = interleaved != 0;
    int i = 0;
    for (int a = 0; a < n_axes; ++a) {
        const int len = ladder == PSA_ROPE_SHARED ? n : sections[a];   // pairs of the ladder
        if (sections[a] == 0) continue;
        const Two y = root(theta, len);
        Two f = ladder == PSA_ROPE_SHARED ? pow2(y, i) : Two{1.0, 0.0};
        for (int k = 0; k < sections[a]; ++k, ++i, f = mul2(f, y)) {
            plan->turn[i] = turns(f);
            plan->axis[i] = (unsigned char)a;
        }
    }
    return ok();
}

int psa_rope(const psa_rope_plan* plan, const psa_attn_view* x, const psa_attn_view* y, int heads, const psa_attn_view* x2,
             const psa_attn_view* y2, int heads2, int B, int N, const int* pos, long long pos_axis_stride,
             long long pos_batch_stride, int inverse, int dtype, void* stream) {
    int rc = check_plan(plan, 0);
    if (rc) return rc;
    if (!dtype_ok(dtype)) return fail(PSA_ERR_ARG, "dtype %d is not PSA_F32 or PSA_BF16", dtype);
    if (!x2 != !y2) return fail(PSA_ERR_ARG, "x2 and y2 are given together or not at all");
    if (!x2) heads2 = 0;
    if (B < 0 || N < 0 || heads < 0 || heads2 < 0)
        return fail(PSA_ERR_ARG, "negative size (B=%d N=%d heads=%d heads2=%d)", B, N, heads, heads2);
    const int d = plan->head_dim;
    if (B == 0 || N == 0 || (heads == 0 && heads2 == 0)) return ok();
    if (N > kMaxRows || (double)B * N * ((double)heads + heads2) * d > (double)kMaxElems)
        return fail(PSA_ERR_UNSUPPORTED, "problem too large (B=%d N=%d heads=%d + %d)", B, N, heads, heads2);
    psa::win::RopeArgs a{};
    a.plan = plan;
    const psa_attn_view* xs[2] = {x, x2};
    const psa_attn_view* ys[2] = {y, y2};
    const int hs[2] = {heads, heads2};
    for (int i = 0; i < 2; ++i) {
        if (i == 0 && !x && heads > 0) return fail(PSA_ERR_ARG, "x view is NULL");
        if (hs[i] == 0) continue;
        if ((rc = check_view(i ? "x2" : "x", xs[i], B, hs[i], N, d, false, &a.x[a.n])) ||
            (rc = check_view(i ? "y2" : "y", ys[i], B, hs[i], N, d, true, &a.y[a.n])))
            return rc;
        a.heads[a.n++] = hs[i];
    }
    if ((rc = check_pos(pos, pos_axis_stride, pos_batch_stride))) return rc;
    a.B = B, a.N = N, a.pos = pos, a.pos_axis = pos_axis_stride, a.pos_batch = pos_batch_stride;
    a.inverse = inverse != 0, a.dtype = dtype, a.stream = (cudaStream_t)stream;
    std::string err;
    rc = psa::win::rope(a, &err);
    return done(rc, err);
}

int psa_win_cache_append(const psa_win_cache* cache, const psa_attn_view* k_new, const psa_attn_view* v_new, int T,
                         const int* start, const int* n_new, const psa_rope_plan* plan, const int* pos,
                         long long pos_axis_stride, long long pos_batch_stride, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (T < 0) return fail(PSA_ERR_ARG, "negative size (T=%d)", T);
    if (plan && (rc = check_plan(plan, cache->head_dim))) return rc;
    if (cache->B == 0 || cache->kv_heads == 0 || T == 0) return ok();
    if (T > kMaxRows || (double)cache->B * T * cache->kv_heads * cache->head_dim > (double)kMaxElems)
        return fail(PSA_ERR_UNSUPPORTED, "problem too large (B=%d T=%d)", cache->B, T);
    psa::win::AppendArgs a{};
    if ((rc = check_view("k_new", k_new, cache->B, cache->kv_heads, T, cache->head_dim, false, &a.kn)) ||
        (rc = check_view("v_new", v_new, cache->B, cache->kv_heads, T, cache->head_dim, false, &a.vn)) ||
        (rc = check_ptr("start", start, 4)) || (rc = check_lens("n_new", n_new)) ||
        (rc = plan ? check_pos(pos, pos_axis_stride, pos_batch_stride) : PSA_OK))
        return rc;
    a.plan = plan, a.k = cache->k, a.v = cache->v, a.B = cache->B, a.Hkv = cache->kv_heads, a.cap = cache->capacity;
    a.d = cache->head_dim, a.sinks = cache->sinks, a.dtype = cache->dtype;
    a.sB = cache->batch_stride, a.sH = cache->head_stride, a.sS = cache->slot_stride;
    a.T = T, a.start = start, a.n_new = n_new, a.pos = pos, a.pos_axis = pos_axis_stride, a.pos_batch = pos_batch_stride;
    a.stream = (cudaStream_t)stream;
    std::string err;
    rc = psa::win::append(a, &err);
    return done(rc, err);
}

size_t psa_win_decode_workspace_bytes(const psa_win_cache* c, int q_heads) {
    const std::string keep = psa_attn_last_error();
    const int rc = check_cache(c);
    psa::set_last_error(rc, keep);
    if (rc || c->B == 0 || c->kv_heads == 0 || q_heads <= 0 || q_heads % c->kv_heads) return 0;
    return psa::win::decode_workspace(c->B, q_heads, c->kv_heads, c->head_dim, c->window, c->sinks, c->dtype);
}

int psa_win_decode(const psa_win_cache* cache, const psa_attn_view* q, const psa_attn_view* o, float* lse, int q_heads,
                   const int* lens, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (q_heads < 0) return fail(PSA_ERR_ARG, "negative size (q_heads=%d)", q_heads);
    if ((cache->kv_heads == 0) != (q_heads == 0) || (cache->kv_heads > 0 && q_heads % cache->kv_heads))
        return fail(PSA_ERR_ARG, "q_heads %d is not a multiple of kv_heads %d", q_heads, cache->kv_heads);
    if (!std::isfinite(scale)) return fail(PSA_ERR_ARG, "scale is not finite");
    if (cache->B == 0 || q_heads == 0) return ok();
    if ((double)cache->B * q_heads * cache->head_dim > (double)kMaxElems)
        return fail(PSA_ERR_UNSUPPORTED, "problem too large (B=%d q_heads=%d)", cache->B, q_heads);
    psa::win::DecodeArgs a{};
    if ((rc = check_view("q", q, cache->B, q_heads, 1, cache->head_dim, false, &a.q)) ||
        (rc = check_view("o", o, cache->B, q_heads, 1, cache->head_dim, true, &a.o)) ||
        (rc = check_ptr("lens", lens, 4)) || (rc = lse ? check_ptr("lse", lse, 4) : PSA_OK))
        return rc;
    const size_t need = psa::win::decode_workspace(cache->B, q_heads, cache->kv_heads, cache->head_dim, cache->window,
                                                   cache->sinks, cache->dtype);
    if (workspace_bytes < need) return fail(PSA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need) {
        if (!workspace) return fail(PSA_ERR_WORKSPACE, "workspace is NULL");
        if ((rc = check_ptr("workspace", workspace, 16))) return rc;
    }
    a.k = cache->k, a.v = cache->v, a.B = cache->B, a.Hq = q_heads, a.Hkv = cache->kv_heads, a.cap = cache->capacity;
    a.d = cache->head_dim, a.window = cache->window, a.sinks = cache->sinks, a.dtype = cache->dtype;
    a.sB = cache->batch_stride, a.sH = cache->head_stride, a.sS = cache->slot_stride;
    a.lse = lse, a.lens = lens, a.scale = scale, a.workspace = workspace, a.stream = (cudaStream_t)stream;
    std::string err;
    rc = psa::win::decode(a, &err);
    return done(rc, err);
}

}  // extern "C"
