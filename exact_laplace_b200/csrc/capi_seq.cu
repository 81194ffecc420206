// capi_seq.cu -- the extern "C" boundary of the sequence operators (declared in
// include/laplex.h): argument checks, workspace carving and the order of the
// passes.  No call allocates, frees, synchronises or throws; host-detected
// errors return before anything is enqueued.
#include <algorithm>

#include "laplex.h"
#include "laplex_impl.h"
#include "seqop.h"

namespace {

#define BAD(...)                       \
    do {                               \
        lx::set_last_error(__VA_ARGS__); \
        return LAPLEX_EINVAL;          \
    } while (0)
#define REQ(cond, ...)             \
    do {                           \
        if (!(cond)) BAD(__VA_ARGS__); \
    } while (0)

constexpr int64_t MAXN = (int64_t)1 << 31;
constexpr int MAX_GROUP = 32, MAX_DIM = 128;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

laplex_status done(cudaError_t e, const char* where) {
    if (e != cudaSuccess) {
        lx::set_last_error("%s: %s", where, cudaGetErrorString(e));
        return LAPLEX_ECUDA;
    }
    lx::set_last_error("%s", "");
    return LAPLEX_OK;
}

bool known_dtype(laplex_dtype d) {
    return d == LAPLEX_F32 || d == LAPLEX_F64 || d == LAPLEX_F16 || d == LAPLEX_BF16;
}

laplex_status check_shape(const laplex_linattn_shape* s, bool step, bool decay) {
    REQ(s != nullptr, "shape is NULL");
    REQ(known_dtype(s->dtype), "dtype %d is not one of the four types", (int)s->dtype);
    REQ(s->tokens >= 0 && s->tokens < MAXN, "tokens = %lld out of range [0, 2^31)", (long long)s->tokens);
    REQ(s->hkv >= 1 && s->hkv <= 65535, "hkv = %d out of range [1, 65535]", s->hkv);
    REQ(s->hq >= 1 && s->hq % s->hkv == 0 && s->hq / s->hkv <= MAX_GROUP,
        "hq = %d is not 1 to %d times hkv = %d", s->hq, MAX_GROUP, s->hkv);
    REQ(s->dk >= 8 && s->dk <= MAX_DIM && s->dk % 8 == 0, "dk = %d is not a multiple of 8 up to %d", s->dk, MAX_DIM);
    REQ(s->dv >= 8 && s->dv <= MAX_DIM && s->dv % 8 == 0, "dv = %d is not a multiple of 8 up to %d", s->dv, MAX_DIM);
    if (!step) {
        REQ(s->seqs >= 0 && s->seqs <= 65535, "seqs = %lld out of range [0, 65535]", (long long)s->seqs);
        REQ(s->seqs > 0 || s->tokens == 0, "no sequences for %lld tokens", (long long)s->tokens);
        if (s->cu_seqlens)
            REQ(aligned(s->cu_seqlens, 4), "cu_seqlens is not aligned");
        else
            REQ(s->seqs == 0 || s->tokens % s->seqs == 0, "cu_seqlens is NULL and seqs = %lld does not divide %lld tokens",
                (long long)s->seqs, (long long)s->tokens);
    }
    if (decay) {
        REQ(s->log_decay != nullptr, "log_decay is NULL");
        REQ(aligned(s->log_decay, lx::acc_bytes(s->dtype)), "log_decay is not aligned");
    }
    return LAPLEX_OK;
}

// Checks an operand and hands it over; the strides of a size of 1 are not read.
laplex_status check_rows(const char* name, const laplex_rows* r, int64_t tokens, int heads, int dim, laplex_dtype dt,
                         bool out, lx::LinRows* to) {
    REQ(r != nullptr, "%s is NULL", name);
    const int64_t es = (int64_t)lx::elem_bytes(dt);
    to->p = r->ptr;
    to->ts = tokens > 1 ? r->token_stride : (int64_t)heads * MAX_DIM;
    to->hs = heads > 1 ? r->head_stride : MAX_DIM;
    if (tokens == 0) return LAPLEX_OK;
    REQ(r->ptr != nullptr, "%s is NULL", name);
    REQ(aligned(r->ptr, 16), "%s is not 16-byte aligned", name);
    if (tokens == 1 && heads > 1) to->ts = std::max<int64_t>(to->ts, heads * to->hs);
    REQ(tokens == 1 || (to->ts >= dim && to->ts * es % 16 == 0 && to->ts < ((int64_t)1 << 36)),
        "%s: token stride %lld", name, (long long)to->ts);
    REQ(heads == 1 || (to->hs >= dim && to->hs * es % 16 == 0 && to->hs < ((int64_t)1 << 36)),
        "%s: head stride %lld", name, (long long)to->hs);
    if (heads == 1) to->hs = MAX_DIM;
    if (out)
        REQ(tokens == 1 || heads == 1 || to->ts >= (heads - 1) * to->hs + dim || to->hs >= (tokens - 1) * to->ts + dim,
            "%s: rows overlap", name);
    return LAPLEX_OK;
}

laplex_status check_state(const char* name, const void* p) {
    REQ(aligned(p, 16), "%s is not 16-byte aligned", name);
    return LAPLEX_OK;
}

#define TRY(x)                                  \
    do {                                        \
        const laplex_status st_ = (x);          \
        if (st_ != LAPLEX_OK) return st_;       \
    } while (0)

lx::LinSeqs make_seqs(const laplex_linattn_shape& s, int seg) {
    lx::LinSeqs S;
    S.cu = s.cu_seqlens;
    S.T = s.tokens;
    S.N = (int)s.seqs;
    S.seg = seg;
    S.slots = s.seqs == 0 ? 0 : (int)(s.tokens / seg + s.seqs);
    return S;
}

bool tensor_cores(const laplex_linattn_shape& s) { return s.dtype == LAPLEX_F16 || s.dtype == LAPLEX_BF16; }

int segment(const laplex_linattn_shape& s, bool backward) {
    const bool equal = s.cu_seqlens == nullptr || s.seqs == 1;
    if (tensor_cores(s)) return lx::tc_segment(s.tokens, (int)s.seqs, s.hkv, backward ? 3 : 1, equal);
    return lx::rec_segment(s.tokens, (int)s.seqs, s.hkv, std::min(s.dk, s.dv), equal);
}

size_t states_bytes(const laplex_linattn_shape& s, int seg) {
    if (seg > s.tokens) return 0;  // no sequence is cut
    return lx::Carve::need((size_t)make_seqs(s, seg).slots * s.hkv * s.dk * s.dv, lx::acc_bytes(s.dtype));
}

size_t linattn_body(const laplex_linattn_shape& s, laplex_linattn_call call) {
    const int seg = segment(s, call != LAPLEX_LINATTN_FORWARD);
    if (call == LAPLEX_LINATTN_FORWARD) return states_bytes(s, seg);
    size_t b = 2 * states_bytes(s, seg);
    if (call == LAPLEX_LINATTN_BACKWARD_DECAY)
        b = std::max(b, lx::dlam_ws_bytes(s.dtype, s.tokens, (int)s.seqs, s.hkv, s.dk, s.dv, s.cu_seqlens == nullptr));
    return b;
}

laplex_status check_ws(void* ws, size_t ws_bytes, size_t body) {
    REQ(ws != nullptr, "workspace is NULL");
    REQ(aligned(ws, 256), "workspace is not 256-byte aligned");
    if (ws_bytes < lx::HEADER_BYTES + body) {
        lx::set_last_error("workspace of %zu bytes, %zu needed", ws_bytes, lx::HEADER_BYTES + body);
        return LAPLEX_EWORKSPACE;
    }
    return LAPLEX_OK;
}

lx::LinRole role(lx::LinRows q, lx::LinRows k, lx::LinRows v, int nq, int nk, int dk, int dv, bool reverse,
                 bool transposed, double sq, double sk) {
    lx::LinRole R = {};
    R.q = q;
    R.k = k;
    R.v = v;
    R.nq = nq;
    R.nk = nk;
    R.dk = dk;
    R.dv = dv;
    R.reverse = reverse;
    R.transposed = transposed;
    R.sq = sq;
    R.sk = sk;
    return R;
}

// The products of roles[0 .. count).  `last`: also the states behind the last tokens, by their own pass.
cudaError_t run(const laplex_linattn_shape& s, const lx::LinRole* roles, int count, const lx::LinRole* last,
                const lx::LinSeqs& S, uint32_t* status, bool next, cudaStream_t st) {
    if (tensor_cores(s)) return lx::tc_run(s.dtype, roles, count, last, S, s.hkv, s.log_decay, status, next, st);
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < count && e == cudaSuccess; ++i)
        e = lx::rec_run(s.dtype, roles[i], S, s.hkv, s.log_decay, false, next || i > 0, st);
    if (e == cudaSuccess && last) e = lx::rec_run(s.dtype, *last, S, s.hkv, s.log_decay, true, next || count > 0, st);
    return e;
}

// The segments' own states alone.
cudaError_t run_states(const laplex_linattn_shape& s, const lx::LinRole* roles, int count, const lx::LinSeqs& S,
                       uint32_t* status, cudaStream_t st) {
    if (tensor_cores(s)) return lx::tc_states(s.dtype, roles, count, S, s.hkv, s.log_decay, status, st);
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < count && e == cudaSuccess; ++i) e = lx::rec_run(s.dtype, roles[i], S, s.hkv, s.log_decay, true, i > 0, st);
    return e;
}

struct Direction {
    lx::LinRole R;
    const void* init;  // per sequence, or NULL
    void* states;      // out, by slot: the states before each segment of R's direction
    void* last;        // out, per sequence: behind the last segment, or NULL
};

cudaError_t segment_states(const laplex_linattn_shape& s, Direction* D, int count, const lx::LinSeqs& S,
                           uint32_t* status, cudaStream_t st) {
    lx::LinRole R[2];
    for (int i = 0; i < count; ++i) {
        R[i] = D[i].R;
        R[i].state_in = nullptr;
        R[i].state_out = D[i].states;
        R[i].out_by_slot = 1;
        R[i].skip_last = D[i].last == nullptr;
        R[i].o = nullptr;
    }
    cudaError_t e = run_states(s, R, count, S, status, st);
    lx::LinCarry C[2] = {};
    for (int i = 0; i < count; ++i) {
        C[i].S = S;
        C[i].H = s.hkv;
        C[i].reverse = D[i].R.reverse;
        C[i].len = (int64_t)s.dk * s.dv;
        C[i].lam = s.log_decay;
        C[i].init = D[i].init;
        C[i].states = D[i].states;
        C[i].last = D[i].last;
    }
    return e == cudaSuccess ? lx::carry_run(s.dtype, C, count, st) : e;
}

}  // namespace

extern "C" {

laplex_status laplex_linattn_workspace_size(const laplex_linattn_shape* shape, laplex_linattn_call call,
                                            size_t* bytes) {
    REQ(bytes != nullptr, "bytes is NULL");
    TRY(check_shape(shape, false, false));
    REQ(call >= LAPLEX_LINATTN_FORWARD && call <= LAPLEX_LINATTN_BACKWARD_DECAY, "unknown call %d", (int)call);
    *bytes = lx::HEADER_BYTES + linattn_body(*shape, call);
    return done(cudaSuccess, "");
}

laplex_status laplex_linattn(const laplex_linattn_shape* shape, const laplex_rows* q, const laplex_rows* k,
                             const laplex_rows* v, const void* state_in, const laplex_rows* o, void* state_out,
                             void* ws, size_t ws_bytes, void* stream) {
    TRY(check_shape(shape, false, true));
    const laplex_linattn_shape& s = *shape;
    lx::LinRows rq, rk, rv, ro;
    TRY(check_rows("q", q, s.tokens, s.hq, s.dk, s.dtype, false, &rq));
    TRY(check_rows("k", k, s.tokens, s.hkv, s.dk, s.dtype, false, &rk));
    TRY(check_rows("v", v, s.tokens, s.hkv, s.dv, s.dtype, false, &rv));
    TRY(check_rows("o", o, s.tokens, s.hq, s.dv, s.dtype, true, &ro));
    TRY(check_state("state_in", state_in));
    TRY(check_state("state_out", state_out));
    TRY(check_ws(ws, ws_bytes, linattn_body(s, LAPLEX_LINATTN_FORWARD)));
    if (s.seqs == 0) return done(cudaSuccess, "");
    cudaStream_t st = (cudaStream_t)stream;
    uint32_t* status = lx::status_word(ws);
    const lx::LinSeqs S = make_seqs(s, segment(s, false));
    lx::LinRole R = role(rq, rk, rv, s.hq / s.hkv, 1, s.dk, s.dv, false, false, s.scale, 1.0);
    R.o = const_cast<void*>(ro.p);
    R.o_ts = ro.ts;
    R.o_hs = ro.hs;
    R.state_in = state_in;
    R.state_out = state_out;
    cudaError_t e = cudaSuccess;
    if (S.seg <= S.T) {
        void* states = static_cast<char*>(ws) + lx::HEADER_BYTES;
        Direction D = {R, state_in, states, state_out};
        e = segment_states(s, &D, 1, S, status, st);
        R.state_in = states;
        R.in_by_slot = 1;
        R.state_out = nullptr;
    }
    // (tensor cores: a state that leaves the call comes from the state pass)
    const bool apart = tensor_cores(s) && R.state_out;
    lx::LinRole P = R;
    if (apart) P.state_out = nullptr;
    if (e == cudaSuccess) e = run(s, &P, 1, apart ? &R : nullptr, S, status, R.in_by_slot, st);
    return done(e, "laplex_linattn");
}

laplex_status laplex_linattn_backward(const laplex_linattn_shape* shape, const laplex_rows* q, const laplex_rows* k,
                                      const laplex_rows* v, const laplex_rows* dout, const void* state_in,
                                      const void* dstate_out, const laplex_rows* dq, const laplex_rows* dk,
                                      const laplex_rows* dv, void* dstate_in, void* dlog_decay, void* ws,
                                      size_t ws_bytes, void* stream) {
    TRY(check_shape(shape, false, true));
    const laplex_linattn_shape& s = *shape;
    lx::LinRows rq, rk, rv, rdo, rdq = {}, rdk = {}, rdv = {};
    TRY(check_rows("q", q, s.tokens, s.hq, s.dk, s.dtype, false, &rq));
    TRY(check_rows("k", k, s.tokens, s.hkv, s.dk, s.dtype, false, &rk));
    TRY(check_rows("v", v, s.tokens, s.hkv, s.dv, s.dtype, false, &rv));
    TRY(check_rows("dout", dout, s.tokens, s.hq, s.dv, s.dtype, false, &rdo));
    if (dq) TRY(check_rows("dq", dq, s.tokens, s.hq, s.dk, s.dtype, true, &rdq));
    if (dk) TRY(check_rows("dk", dk, s.tokens, s.hkv, s.dk, s.dtype, true, &rdk));
    if (dv) TRY(check_rows("dv", dv, s.tokens, s.hkv, s.dv, s.dtype, true, &rdv));
    TRY(check_state("state_in", state_in));
    TRY(check_state("dstate_out", dstate_out));
    TRY(check_state("dstate_in", dstate_in));
    REQ(dstate_in == nullptr || (dstate_in != dstate_out && dstate_in != state_in), "dstate_in overlaps an input");
    REQ(aligned(dlog_decay, lx::acc_bytes(s.dtype)), "dlog_decay is not aligned");
    TRY(check_ws(ws, ws_bytes, linattn_body(s, dlog_decay ? LAPLEX_LINATTN_BACKWARD_DECAY : LAPLEX_LINATTN_BACKWARD)));
    cudaStream_t st = (cudaStream_t)stream;
    char* body = static_cast<char*>(ws) + lx::HEADER_BYTES;
    const int G = s.hq / s.hkv;
    uint32_t* status = lx::status_word(ws);
    const lx::LinSeqs S = make_seqs(s, segment(s, true));
    cudaError_t e = cudaSuccess;
    if (dlog_decay) {
        lx::LinRole R = role(rq, rk, rv, G, 1, s.dk, s.dv, false, false, s.scale, 1.0);
        e = lx::dlam_run(s.dtype, R, rdo, S, s.hkv, s.log_decay, state_in, dstate_out, dlog_decay, body,
                         ws_bytes - lx::HEADER_BYTES, st);
        if (e != cudaSuccess) return done(e, "laplex_linattn_backward");
    }
    if (s.seqs == 0) return done(cudaSuccess, "");
    lx::LinRole Rq = role(rdo, rv, rk, G, 1, s.dv, s.dk, false, true, s.scale, 1.0);
    lx::LinRole Rk = role(rv, rdo, rq, 1, G, s.dv, s.dk, true, true, 1.0, s.scale);
    lx::LinRole Rv = role(rk, rq, rdo, 1, G, s.dk, s.dv, true, false, 1.0, s.scale);
    const bool rev = dk || dv || dstate_in;
    Rq.state_in = state_in;
    Rk.state_in = Rv.state_in = dstate_out;
    const bool cut = S.seg <= S.T;
    if (cut) {
        void* fwd = body;
        void* bwd = body + states_bytes(s, S.seg);
        Direction D[2];
        int count = 0;
        if (dq) D[count++] = {role(rq, rk, rv, G, 1, s.dk, s.dv, false, false, s.scale, 1.0), state_in, fwd, nullptr};
        if (rev) D[count++] = {Rv, dstate_out, bwd, dstate_in};
        e = segment_states(s, D, count, S, status, st);
        if (e != cudaSuccess) return done(e, "laplex_linattn_backward");
        Rq.state_in = fwd;
        Rk.state_in = Rv.state_in = bwd;
        Rq.in_by_slot = Rk.in_by_slot = Rv.in_by_slot = 1;
    }
    const auto out = [](lx::LinRole* R, const lx::LinRows& to) {
        R->o = const_cast<void*>(to.p);
        R->o_ts = to.ts;
        R->o_hs = to.hs;
    };
    lx::LinRole roles[3];
    int count = 0;
    if (dq) {
        out(&Rq, rdq);
        roles[count++] = Rq;
    }
    if (dk) {
        out(&Rk, rdk);
        roles[count++] = Rk;
    }
    const bool apart = dstate_in && !cut && (tensor_cores(s) || !dv);
    if (!cut && !apart) Rv.state_out = dstate_in;
    if (dv) {
        out(&Rv, rdv);
        roles[count++] = Rv;
    }
    Rv.state_out = dstate_in;
    e = run(s, roles, count, apart ? &Rv : nullptr, S, status, cut, st);
    return done(e, "laplex_linattn_backward");
}

laplex_status laplex_test_set_linattn_wait(uint32_t polls, int force_expiry) {
    lx::set_linattn_wait(polls, force_expiry);
    return done(cudaSuccess, "");
}

laplex_status laplex_linattn_step(const laplex_linattn_shape* shape, const laplex_rows* q, const laplex_rows* k,
                                  const laplex_rows* v, void* states, int64_t num_slots, const int32_t* slots,
                                  const laplex_rows* o, void* stream) {
    TRY(check_shape(shape, true, true));
    const laplex_linattn_shape& s = *shape;
    lx::LinRows rq, rk, rv, ro;
    TRY(check_rows("q", q, s.tokens, s.hq, s.dk, s.dtype, false, &rq));
    TRY(check_rows("k", k, s.tokens, s.hkv, s.dk, s.dtype, false, &rk));
    TRY(check_rows("v", v, s.tokens, s.hkv, s.dv, s.dtype, false, &rv));
    TRY(check_rows("o", o, s.tokens, s.hq, s.dv, s.dtype, true, &ro));
    REQ(num_slots >= 0 && num_slots < MAXN, "num_slots = %lld out of range [0, 2^31)", (long long)num_slots);
    REQ(states != nullptr || num_slots == 0, "states is NULL");
    TRY(check_state("states", states));
    REQ(slots != nullptr || s.tokens <= num_slots, "%lld rows for %lld states", (long long)s.tokens, (long long)num_slots);
    REQ(aligned(slots, 4), "slots is not aligned");
    lx::LinStep P;
    P.q = rq;
    P.k = rk;
    P.v = rv;
    P.o = const_cast<void*>(ro.p);
    P.o_ts = ro.ts;
    P.o_hs = ro.hs;
    P.rows = s.tokens;
    P.slots = num_slots;
    P.hq = s.hq;
    P.hkv = s.hkv;
    P.dk = s.dk;
    P.dv = s.dv;
    P.slot = slots;
    P.lam = s.log_decay;
    P.scale = s.scale;
    P.states = states;
    return done(lx::step_run(s.dtype, P, (cudaStream_t)stream), "laplex_linattn_step");
}

static laplex_status check_embed(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt) {
    REQ(known_dtype(dt), "dtype %d is not one of the four types", (int)dt);
    REQ(n >= 0 && n < MAXN, "n = %lld out of range [0, 2^31)", (long long)n);
    REQ(rows >= 0 && rows < MAXN, "rows = %lld out of range [0, 2^31)", (long long)rows);
    REQ(dim >= 1 && dim < MAXN, "dim = %lld out of range [1, 2^31)", (long long)dim);
    return LAPLEX_OK;
}

static laplex_status check_table(const char* name, const void* p, int64_t rows, int64_t ld, int64_t dim) {
    REQ(rows == 0 || p != nullptr, "%s is NULL", name);
    REQ(aligned(p, 16), "%s is not 16-byte aligned", name);
    REQ(rows <= 1 || (ld >= dim && ld < ((int64_t)1 << 36)), "%s: row stride %lld", name, (long long)ld);
    return LAPLEX_OK;
}

static laplex_status check_tokens(const void* tokens, int token_bytes, int64_t n) {
    REQ(token_bytes == 4 || token_bytes == 8, "token_bytes = %d is not 4 or 8", token_bytes);
    REQ(n == 0 || tokens != nullptr, "tokens is NULL");
    REQ(aligned(tokens, (size_t)token_bytes), "tokens is not aligned");
    return LAPLEX_OK;
}

laplex_status laplex_embed(const void* table, int64_t ld, int64_t rows, int64_t dim, const void* tokens,
                           int token_bytes, int64_t n, double scale, void* out, int64_t out_ld, laplex_dtype dt,
                           void* stream) {
    TRY(check_embed(n, rows, dim, dt));
    TRY(check_tokens(tokens, token_bytes, n));
    TRY(check_table("table", table, rows, ld, dim));
    TRY(check_table("out", out, n, out_ld, dim));
    lx::EmbedArgs A = {};
    A.tokens = tokens;
    A.tok64 = token_bytes == 8;
    A.n = n;
    A.rows = rows;
    A.dim = dim;
    A.src = table;
    A.src_ld = rows > 1 ? ld : 0;
    A.dst = out;
    A.dst_ld = n > 1 ? out_ld : 0;
    A.scale = scale;
    return done(lx::embed_run(dt, A, (cudaStream_t)stream), "laplex_embed");
}

laplex_status laplex_embed_backward_workspace_size(int64_t n, int64_t rows, int64_t dim, laplex_dtype dt,
                                                   size_t* bytes) {
    REQ(bytes != nullptr, "bytes is NULL");
    TRY(check_embed(n, rows, dim, dt));
    *bytes = lx::HEADER_BYTES + lx::embed_bwd_ws_bytes(n, rows, dim, dt);
    return done(cudaSuccess, "");
}

laplex_status laplex_embed_backward(const void* tokens, int token_bytes, int64_t n, const void* g, int64_t g_ld,
                                    int64_t rows, int64_t dim, double scale, int accumulate, void* dtable, int64_t ld,
                                    laplex_dtype dt, laplex_dtype out_dt, void* ws, size_t ws_bytes, void* stream) {
    TRY(check_embed(n, rows, dim, dt));
    REQ(out_dt == dt || (out_dt == LAPLEX_F32 && dt != LAPLEX_F64), "out_dtype %d is neither dtype nor LAPLEX_F32", (int)out_dt);
    TRY(check_tokens(tokens, token_bytes, n));
    TRY(check_table("g", g, n, g_ld, dim));
    TRY(check_table("dtable", dtable, rows, ld, dim));
    TRY(check_ws(ws, ws_bytes, lx::embed_bwd_ws_bytes(n, rows, dim, dt)));
    lx::EmbedArgs A = {};
    A.tokens = tokens;
    A.tok64 = token_bytes == 8;
    A.n = n;
    A.rows = rows;
    A.dim = dim;
    A.src = g;
    A.src_ld = n > 1 ? g_ld : 0;
    A.dst = dtable;
    A.dst_ld = rows > 1 ? ld : 0;
    A.scale = scale;
    A.accumulate = accumulate != 0;
    return done(lx::embed_bwd_run(dt, out_dt, A, static_cast<char*>(ws) + lx::HEADER_BYTES, ws_bytes - lx::HEADER_BYTES,
                                  lx::status_word(ws), (cudaStream_t)stream),
                "laplex_embed_backward");
}

}  // extern "C"
