// Host front end of the logit operators declared in include/ccl.h: argument
// and alias checks, and the dispatch to their kernels.
#include "ccl.h"

#include <cuda_runtime.h>

#include "front.h"

using namespace ccl;

// A buffer beside the rank buffers: what it is called, where it lies, whether
// the call writes it.
struct Aux {
    const char *name;
    Range at;
    bool written;
};

// A rank buffer: `rows` pieces of `width` bytes, `stride` bytes apart; bytes from the first to the last of them.
struct Shape {
    uint64_t rows = 0, width = 0, stride = 0;
    uint64_t extent() const { return rows && width ? (rows - 1) * stride + width : 0; }
};

// Whether two buffers whose ranges overlap have a byte in common.  Rows of one
// stride may lie between one another's, as the columns of one matrix do.
static bool rows_meet(uintptr_t pa, const Shape &a, uintptr_t pb, const Shape &b)
{
    if (a.rows != b.rows || a.stride != b.stride || a.rows < 2) return true;
    // b's row i + k begins d + k stride behind a's row i: the least k for which it ends behind the latter's begin
    const int64_t d = int64_t(pb - pa), s = int64_t(a.stride), last = int64_t(a.rows) - 1;
    const int64_t n = -int64_t(b.width) - d;
    int64_t k = n / s - (n % s < 0 ? 1 : 0) + 1;
    if (k < -last) k = -last;
    return k <= last && d + k * s < int64_t(a.width);
}

// Rank buffers: aligned to their elements; where the call writes the outputs,
// each is its own rank's input or disjoint from every input and every other
// output.  What the call writes beside them overlaps nothing, and nothing it
// reads overlaps an output.  *alias: every output that has elements is its
// rank's input; where that holds for some ranks alone, a kernel has to write
// all of each output.
static ccl_status_t check_buffers(const ccl_comm *c, const Shape *shape, size_t es, bool outputs, const Aux *aux, int n_aux,
                                  bool *alias)
{
    const int p = c->p;
    Range in[kMaxRanks], out[kMaxRanks];
    *alias = outputs;
    for (int r = 0; r < p; ++r) {
        in[r] = range_of(c->in[r], shape[r].extent());
        out[r] = range_of(c->out[r], shape[r].extent());
        if (in[r].lo < in[r].hi && out[r].lo != in[r].lo) *alias = false;
        if (uintptr_t(c->in[r]) % es || (outputs && uintptr_t(c->out[r]) % es))
            return fail(CCL_ERR_INVALID_ARG, "a buffer of rank %d is not aligned to its elements (%zu bytes)", r, es);
    }
    for (int k = 0; outputs && k < p; ++k) {
        for (int j = 0; j < p; ++j) {
            if (j > k && overlap(out[k], out[j]) && rows_meet(out[k].lo, shape[k], out[j].lo, shape[j]))
                return fail(CCL_ERR_INVALID_ARG, "outputs of ranks %d and %d overlap", k, j);
            if (overlap(out[k], in[j]) && (j != k || out[k].lo != in[k].lo) && rows_meet(out[k].lo, shape[k], in[j].lo, shape[j]))
                return fail(CCL_ERR_INVALID_ARG, "output of rank %d overlaps the input of rank %d", k, j);
        }
    }
    for (int i = 0; i < n_aux; ++i) {
        for (int r = 0; r < p; ++r) {
            if (outputs && overlap(aux[i].at, out[r]))
                return fail(CCL_ERR_INVALID_ARG, "%s overlaps the output of rank %d", aux[i].name, r);
            if (aux[i].written && overlap(aux[i].at, in[r]))
                return fail(CCL_ERR_INVALID_ARG, "%s overlaps the input of rank %d", aux[i].name, r);
        }
        for (int j = 0; aux[i].written && j < n_aux; ++j)
            if (j != i && overlap(aux[i].at, aux[j].at))
                return fail(CCL_ERR_INVALID_ARG, "%s overlaps %s", aux[i].name, aux[j].name);
    }
    return CCL_OK;
}

// [rows, vocab] logits over the ranks' shards: the shape of each shard.
static ccl_status_t shard_shapes(const ccl_comm *c, size_t rows, size_t vocab, size_t ld, size_t es, Shape *shape)
{
    if (vocab == 0 || vocab > (size_t(1) << 30)) return fail(CCL_ERR_INVALID_ARG, "vocab %zu outside [1, 2^30]", vocab);
    if (rows > 0x7fffffffull) return fail(CCL_ERR_INVALID_ARG, "rows %zu above 2^31 - 1", rows);
    uint64_t bound[kMaxRanks + 1];
    chunk_bounds(c->p, vocab, bound);
    if (ld && ld < bound[1]) return fail(CCL_ERR_INVALID_ARG, "ld %zu below the widest shard, %llu", ld, (unsigned long long)bound[1]);
    const uint64_t widest = ld ? ld : bound[1];
    if (rows && widest > (SIZE_MAX / 4) / rows / es) return fail(CCL_ERR_INVALID_ARG, "rows * columns too large");
    for (int r = 0; r < c->p; ++r) {
        const uint64_t w = bound[r + 1] - bound[r];
        shape[r] = {rows, w * es, (ld ? ld : w) * es};
    }
    return CCL_OK;
}

static const char *kPassName[] = {"-", "forward", "backward", "both"};

extern "C" ccl_status_t ccl_logit_rules(ccl_comm_t c, ccl_dtype_t dtype, size_t rows, size_t vocab, size_t ld,
                                        const ccl_logit_rules_t *rules, void *stream)
{
    ccl_status_t st = check_floats(c, dtype, "ccl_logit_rules");
    if (st != CCL_OK) return st;
    if (!rules) return fail(CCL_ERR_INVALID_ARG, "rules is NULL");
    Shape shape[kMaxRanks];
    const size_t es = elem_bytes(dtype);
    st = shard_shapes(c, rows, vocab, ld, es, shape);
    if (st != CCL_OK) return st;
    if (rows == 0) return CCL_OK;
    ccl_logit_rules_t r = *rules;
    const bool penalised = r.repetition || r.frequency || r.presence;
    if (!r.history && r.history_ld) return fail(CCL_ERR_INVALID_ARG, "history_ld %zu with a NULL history", r.history_ld);
    if (r.history_ld > 0x3fffffffull) return fail(CCL_ERR_INVALID_ARG, "history_ld %zu above 2^30 - 1", r.history_ld);
    if (!penalised || r.history_ld == 0) r.history = nullptr;   // a history that nothing weighs
    if (r.bias_count > 0x7fffffffull) return fail(CCL_ERR_INVALID_ARG, "bias_count %zu above 2^31 - 1", r.bias_count);
    if (r.bias_count && (!r.bias_offsets || !r.bias_tokens || !r.bias_values))
        return fail(CCL_ERR_INVALID_ARG, "bias_count %zu with a NULL bias array", r.bias_count);
    const size_t words = (vocab + 31) / 32;
    if (r.mask && r.mask_ld < words) return fail(CCL_ERR_INVALID_ARG, "mask_ld %zu below %zu words", r.mask_ld, words);
    if (r.mask && !r.mask_index && r.mask_rows < rows)
        return fail(CCL_ERR_INVALID_ARG, "mask_rows %zu below rows %zu without a mask_index", r.mask_rows, rows);
    if (r.mask && r.mask_rows && r.mask_ld > (SIZE_MAX / 8) / r.mask_rows) return fail(CCL_ERR_INVALID_ARG, "mask too large");
    if (r.mask_rows == 0) r.mask = nullptr;
    const Aux aux[] = {
        {"repetition", range_of(r.repetition, rows * 4), false},
        {"frequency", range_of(r.frequency, rows * 4), false},
        {"presence", range_of(r.presence, rows * 4), false},
        {"history", range_of(r.history, rows * r.history_ld * 4), false},
        {"history_len", range_of(r.history_len, rows * 4), false},
        {"prompt_len", range_of(r.prompt_len, rows * 4), false},
        {"bias_offsets", range_of(r.bias_count ? r.bias_offsets : nullptr, (rows + 1) * 4), false},
        {"bias_tokens", range_of(r.bias_count ? r.bias_tokens : nullptr, r.bias_count * 4), false},
        {"bias_values", range_of(r.bias_count ? r.bias_values : nullptr, r.bias_count * 4), false},
        {"mask", range_of(r.mask, r.mask ? ((r.mask_rows - 1) * r.mask_ld + words) * 4 : 0), false},
        {"mask_index", range_of(r.mask ? r.mask_index : nullptr, rows * 4), false},
    };
    for (const Aux &a : aux)
        if (a.at.lo % 4) return fail(CCL_ERR_INVALID_ARG, "%s is not aligned to its elements (4 bytes)", a.name);
    bool alias = false;
    st = check_buffers(c, shape, es, true, aux, int(sizeof aux / sizeof aux[0]), &alias);
    if (st != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "logit_rules");
    RulesLaunch N;
    N.rows = rows;
    N.vocab = uint32_t(vocab);
    N.ld = ld;
    N.rules = &r;
    LaunchInfo info;
    const cudaError_t err = launch_logit_rules(make_launch(c, dtype, alias, stream), N, &info);
    return finish(c, err, info, dtype, rows, vocab, "logit_rules", kPassName[0]);
}

extern "C" ccl_status_t ccl_distill_topk(ccl_comm_t c, ccl_dtype_t dtype, ccl_pass_t pass, size_t rows, size_t vocab, size_t ld,
                                         size_t k, const int32_t *teacher_ids, const void *teacher_logits,
                                         ccl_dtype_t teacher_dtype, float temperature, const float *row_weight, float *loss,
                                         float *stats, void *stream)
{
    ccl_status_t st = check_floats(c, dtype, "ccl_distill_topk");
    if (st != CCL_OK) return st;
    if (pass < CCL_PASS_FORWARD || pass > CCL_PASS_BOTH) return fail(CCL_ERR_INVALID_ARG, "unknown pass %d", int(pass));
    if (teacher_dtype < CCL_F32 || teacher_dtype > CCL_BF16)
        return fail(CCL_ERR_INVALID_ARG, "teacher_dtype %d is not a floating-point type", int(teacher_dtype));
    if (!(temperature > 0.0f) || temperature > 3.0e38f) return fail(CCL_ERR_INVALID_ARG, "temperature must be finite and > 0");
    if (temperature < 4.25e-39f)     // log2(e) / temperature would not be finite, and 0 times it not 0
        return fail(CCL_ERR_INVALID_ARG, "temperature %g below 4.25e-39: its reciprocal leaves fp32's range", double(temperature));
    if (k == 0) return fail(CCL_ERR_INVALID_ARG, "k must be positive");
    if (k > 1024) return fail(CCL_ERR_UNSUPPORTED, "k=%zu above 1024 teacher entries a row", k);
    Shape shape[kMaxRanks];
    const size_t es = elem_bytes(dtype), ts = elem_bytes(teacher_dtype);
    st = shard_shapes(c, rows, vocab, ld, es, shape);
    if (st != CCL_OK) return st;
    if (rows == 0) return CCL_OK;
    const bool fwd = pass & CCL_PASS_FORWARD, bwd = pass & CCL_PASS_BACKWARD;
    if (!teacher_ids || !teacher_logits) return fail(CCL_ERR_INVALID_ARG, "NULL teacher_ids or teacher_logits");
    if (fwd && !loss) return fail(CCL_ERR_INVALID_ARG, "the forward pass needs loss");
    if (!fwd && !stats) return fail(CCL_ERR_INVALID_ARG, "the backward pass needs the forward pass's stats");
    if (!fwd) loss = nullptr;
    if (!bwd) row_weight = nullptr;
    const Aux aux[] = {
        {"teacher_ids", range_of(teacher_ids, rows * k * 4), false},
        {"teacher_logits", range_of(teacher_logits, rows * k * ts), false},
        {"row_weight", range_of(row_weight, rows * 4), false},
        {"loss", range_of(loss, rows * 4), fwd},
        {"stats", range_of(stats, rows * 8), fwd},
    };
    for (int i = 0; i < 5; ++i)
        if ((st = check_aligned(reinterpret_cast<const void *>(aux[i].at.lo), i == 1 ? ts : 4, aux[i].name)) != CCL_OK) return st;
    bool alias = false;
    st = check_buffers(c, shape, es, bwd, aux, 5, &alias);
    if (st != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "distill_topk");
    DistillLaunch N;
    N.pass = pass;
    N.rows = rows;
    N.vocab = uint32_t(vocab);
    N.ld = ld;
    N.k = uint32_t(k);
    N.ids = teacher_ids;
    N.teacher = teacher_logits;
    N.teacher_dtype = teacher_dtype;
    N.temperature = temperature;
    N.weight = row_weight;
    N.loss = loss;
    N.stats = stats;
    LaunchInfo info;
    const cudaError_t err = launch_distill(make_launch(c, dtype, alias, stream), N, &info);
    return finish(c, err, info, dtype, rows, vocab, "distill_topk", kPassName[pass]);
}

extern "C" ccl_status_t ccl_balance_loss(ccl_comm_t c, ccl_dtype_t dtype, ccl_pass_t pass, size_t rows, size_t experts, size_t k,
                                         const int32_t *const *expert_ids, const uint8_t *const *valid, float coef,
                                         const float *dloss, int32_t *counts, int32_t *tokens, float *loss, void *stream)
{
    ccl_status_t st = check_floats(c, dtype, "ccl_balance_loss");
    if (st != CCL_OK) return st;
    if (pass < CCL_PASS_FORWARD || pass > CCL_PASS_BOTH) return fail(CCL_ERR_INVALID_ARG, "unknown pass %d", int(pass));
    if (experts == 0) return fail(CCL_ERR_INVALID_ARG, "experts must be positive");
    if (experts > 4096) return fail(CCL_ERR_UNSUPPORTED, "experts=%zu above 4096", experts);
    if (k == 0 || k > experts) return fail(CCL_ERR_INVALID_ARG, "k=%zu outside [1, %zu]", k, experts);
    if (rows > 0x7fffffffull / k) return fail(CCL_ERR_INVALID_ARG, "rows * k above 2^31 - 1: a rank's counts are 32-bit");
    if (!(coef >= -3.0e38f && coef <= 3.0e38f)) return fail(CCL_ERR_INVALID_ARG, "coef must be finite");
    const bool fwd = pass & CCL_PASS_FORWARD, bwd = pass & CCL_PASS_BACKWARD;
    if (rows == 0 && !fwd) return CCL_OK;
    const int p = c->p;
    const size_t es = elem_bytes(dtype);
    if (!counts || !tokens) return fail(CCL_ERR_INVALID_ARG, "NULL counts or tokens");
    if (fwd && !loss) return fail(CCL_ERR_INVALID_ARG, "the forward pass needs loss");
    if (fwd && !expert_ids) return fail(CCL_ERR_INVALID_ARG, "the forward pass needs expert_ids");
    for (int r = 0; r < p; ++r) {
        if (fwd && !expert_ids[r]) return fail(CCL_ERR_INVALID_ARG, "expert_ids[%d] is NULL", r);
        if (valid && !valid[r]) return fail(CCL_ERR_INVALID_ARG, "valid[%d] is NULL", r);
    }
    if (!fwd) {
        expert_ids = nullptr;
        loss = nullptr;
    }
    if (!bwd) dloss = nullptr;
    Aux aux[4 + 2 * kMaxRanks];
    int n = 0;
    aux[n++] = {"counts", range_of(counts, size_t(p) * experts * 4), fwd};
    aux[n++] = {"tokens", range_of(tokens, size_t(p) * 4), fwd};
    aux[n++] = {"loss", range_of(loss, 4), fwd};
    aux[n++] = {"dloss", range_of(dloss, 4), false};
    for (int r = 0; r < p; ++r) {
        if (expert_ids) aux[n++] = {"expert_ids", range_of(expert_ids[r], rows * k * 4), false};
        if (valid) aux[n++] = {"valid", range_of(valid[r], rows), false};
    }
    for (int i = 0; i < n; ++i)
        if (aux[i].name[0] != 'v' && (st = check_aligned(reinterpret_cast<const void *>(aux[i].at.lo), 4, aux[i].name)) != CCL_OK) return st;
    Shape shape[kMaxRanks];
    for (int r = 0; r < p; ++r) shape[r] = {rows, experts * es, experts * es};
    bool alias = false;
    st = check_buffers(c, shape, es, bwd, aux, n, &alias);
    if (st != CCL_OK) return st;
    DeviceGuard g(c->device);
    if (g.err != cudaSuccess) return cuda_fail(g.err, "balance_loss");
    BalanceLaunch N;
    N.pass = pass;
    N.rows = rows;
    N.experts = uint32_t(experts);
    N.k = uint32_t(k);
    N.ids = expert_ids;
    N.valid = valid;
    N.coef = coef;
    N.dloss = dloss;
    N.counts = counts;
    N.tokens = tokens;
    N.loss = loss;
    N.scratch = reinterpret_cast<char *>(c->d_status) + kScratchOffset;
    LaunchInfo info;
    const cudaError_t err = launch_balance(make_launch(c, dtype, alias, stream), N, &info);
    return finish(c, err, info, dtype, rows, experts, "balance_loss", kPassName[pass]);
}
