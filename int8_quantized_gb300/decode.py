"""One attention layer of a quantized decoder, a token per sequence at a time:

  x -> QGemmDyn or MatMulNBits (q, k and v)
    -> kv_append (norms of the heads, rotary positions, int8 pages)
    -> paged_attention (weights added to the scores)
    -> QGemmDyn or MatMulNBits (output)

and, when a sequence reaches its capacity, kv_evict into fresh pages.  TokenHead
turns the last layer's output into tokens: MatMulNBits (logits) -> sample.  Run
as a module it decodes a few tokens with random weights of 4 bits:

    python -m int8_quantized_gb300.decode
"""
import torch

import int8_quantized_gb300 as q


class DecodeAttention:
    """Weights are int8 [in, out] with a scale per output column (typeB
    I8Q_S8 of QGemmDyn): w_qkv [hidden, (q_heads + 2 kv_heads) * head_dim],
    w_out [q_heads * head_dim, hidden]; or MatMulNBits of those products, and
    None for their scales.  cos, sin: fp32 [positions, pairs].  q_norm,
    k_norm [head_dim], norm_eps: as kv_append's.

    A sequence that holds `capacity` tokens is cut to `budget` before its next
    token: the first `sink`, the last `recent` and the most attended others.
    """

    def __init__(self, w_qkv, w_qkv_scale, w_out, w_out_scale, cos, sin, *, sequences, q_heads, kv_heads, head_dim,
                 capacity, budget, sink=4, recent=32, page_size=16, q_norm=None, k_norm=None, norm_eps=1e-6):
        if not 0 < budget < capacity:
            raise ValueError("budget must be below capacity")
        if sink < 0 or recent < 0 or sink + recent > budget:
            raise ValueError("sink + recent must be within 0 .. budget")
        dev = w_qkv.device
        if isinstance(w_qkv, q.MatMulNBits):
            hidden, width = w_qkv.K, w_qkv.N
        else:
            hidden, width = w_qkv.shape
        if width != (q_heads + 2 * kv_heads) * head_dim:
            raise ValueError(f"w_qkv must have {(q_heads + 2 * kv_heads) * head_dim} outputs, it has {width}")
        self.norms = dict(q_norm=q_norm, k_norm=k_norm, norm_eps=norm_eps)
        self.B, self.Hq, self.H, self.D = sequences, q_heads, kv_heads, head_dim
        self.capacity, self.budget, self.sink, self.recent, self.page = capacity, budget, sink, recent, page_size
        self.qkv_gemm = self._product(w_qkv, w_qkv_scale, sequences, width, hidden)
        self.out_gemm = self._product(w_out, w_out_scale, sequences, hidden, q_heads * head_dim)
        self.cos, self.sin = cos, sin
        per = -(-capacity // page_size)
        pages = sequences * per + -(-budget // page_size)  # one sequence at a time moves into the spare pages
        shape = (pages, kv_heads, page_size, head_dim)
        k, scale = torch.zeros(shape, dtype=torch.int8, device=dev), torch.ones(shape[:3], device=dev)
        self.cache = q.KVCache(k, torch.zeros_like(k), scale, scale.clone(), torch.zeros_like(scale))
        self.free = list(range(pages))
        self.table = torch.full((sequences, per), -1, dtype=torch.int32, device=dev)
        self.owned = [[] for _ in range(sequences)]
        self.length = [0] * sequences
        self.position = [0] * sequences                # of the next token; eviction does not change it
        self.seq = torch.arange(sequences, dtype=torch.int32, device=dev)
        self.qkv = torch.empty((sequences, width), dtype=torch.bfloat16, device=dev)
        self.attended = torch.empty((sequences, q_heads, head_dim), dtype=torch.bfloat16, device=dev)
        self.workspace = torch.empty(q.paged_attention_workspace_size(self.cache, self.table, q_heads, True),
                                     dtype=torch.uint8, device=dev)

    @staticmethod
    def _product(weight, scale, rows, outputs, depth):
        if isinstance(weight, q.MatMulNBits):
            if (weight.N, weight.K) != (outputs, depth):
                raise ValueError(f"a matrix of {weight.K} to {weight.N} where {depth} to {outputs} are needed")
            return weight
        gemm = q.QGemmDyn(rows, outputs, depth, q.BF16, q.S8, q.BF16, bias=False)
        gemm.set_params(weight, scale)
        return gemm

    def _grow(self, b):
        if self.length[b] == len(self.owned[b]) * self.page:
            self.owned[b].append(self.free.pop())
            self.table[b, len(self.owned[b]) - 1] = self.owned[b][-1]

    def evict(self, b):
        """Cut sequence b to its budget; returns the kept tokens' indices [kv_heads, budget]."""
        dev = self.table.device
        need = -(-self.budget // self.page)
        new = self.free[-need:]
        new_table = torch.tensor([new], dtype=torch.int32, device=dev)
        kept = torch.empty((1, self.H, self.budget), dtype=torch.int32, device=dev)
        q.kv_evict(self.cache, self.table[b:b + 1], torch.tensor([self.length[b]], dtype=torch.int32, device=dev),
                   new_table, kept, sink=self.sink, recent=self.recent)
        self.free = self.free[:-need] + self.owned[b]
        self.owned[b], self.length[b] = new, min(self.length[b], self.budget)
        self.table[b].fill_(-1)
        self.table[b, :need] = new_table[0]
        return kept[0]

    def step(self, x, out):
        """x, out: bf16 [sequences, hidden], the next token of every sequence."""
        dev = x.device
        if max(self.position) >= self.cos.shape[0]:
            raise ValueError("a sequence has no position left in cos and sin")
        for b in range(self.B):
            if self.length[b] == self.capacity:
                self.evict(b)
            self._grow(b)
        self.qkv_gemm.forward(x, self.qkv)
        rows = self.qkv.view(self.B, self.Hq + 2 * self.H, self.D)
        query, key, value = rows.split((self.Hq, self.H, self.H), 1)
        index = torch.tensor(self.length, dtype=torch.int32, device=dev)
        positions = torch.tensor(self.position, dtype=torch.int32, device=dev)
        q.kv_append(self.cache, self.table, self.seq, index, key, value, q=query, q_out=query, positions=positions,
                    cos=self.cos, sin=self.sin, **self.norms)
        q.paged_attention(self.cache, self.table, index + 1, query, self.attended, accumulate=True,
                          workspace=self.workspace)
        self.out_gemm.forward(self.attended.view(self.B, -1), out)
        self.length = [n + 1 for n in self.length]
        self.position = [n + 1 for n in self.position]
        return out


class TokenHead:
    """The next tokens from the last layer's output: logits of a MatMulNBits
    `head` [hidden to vocabulary], then sample with the given settings (None, or
    a tensor of `sequences` entries, as sample's)."""

    def __init__(self, head, sequences, temperature=None, top_k=None, top_p=None, min_p=None):
        self.head = head
        self.settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        self.logits = torch.empty((sequences, head.N), dtype=torch.bfloat16, device=head.device)
        self.tokens = torch.empty((sequences,), dtype=torch.int32, device=head.device)
        self.logprobs = torch.empty((sequences,), dtype=torch.float32, device=head.device)

    def step(self, x, random):
        """x bf16 [sequences, hidden], random fp32 [sequences] in [0, 1): the
        tokens int32 [sequences]; their logarithms stand in logprobs."""
        self.head.forward(x, self.logits)
        return q.sample(self.logits, random, self.tokens, logprobs=self.logprobs, **self.settings)


def random_nbits(rows, columns, g, device="cuda", block_size=64):
    """A MatMulNBits [rows to columns] of random codes, its outputs about as large as its inputs."""
    blocks = -(-rows // block_size)
    codes = torch.randint(0, 256, (columns, blocks, block_size // 2), generator=g, device=device, dtype=torch.uint8)
    scales = torch.full((columns, blocks), 1.0 / (4.6 * rows ** 0.5), device=device).to(torch.bfloat16)
    return q.MatMulNBits(codes, scales, rows, block_size)


def random_layer(sequences=4, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, capacity=96, budget=64, positions=4096,
                 seed=0, device="cuda", sink=None, recent=None, bits=8, norms=False):
    """A DecodeAttention with random weights of 8 or 4 bits, with or without norms of the heads of q and k; sink and
    recent: 4 and 32, or what the budget has room for."""
    sink = min(4, budget) if sink is None else sink
    recent = min(32, budget - sink) if recent is None else recent
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def weight(rows, columns):
        if bits == 4:
            return random_nbits(rows, columns, g, device), None
        w = torch.randint(-127, 128, (rows, columns), generator=g, device=device, dtype=torch.int8)
        return w, torch.full((columns,), 1.0 / (73.0 * rows ** 0.5), device=device)

    pairs = head_dim // 2
    turn = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs) / pairs)
    return DecodeAttention(*weight(hidden, (q_heads + 2 * kv_heads) * head_dim), *weight(q_heads * head_dim, hidden),
                           turn.cos().float().to(device), turn.sin().float().to(device), sequences=sequences,
                           q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, capacity=capacity, budget=budget,
                           sink=sink, recent=recent, q_norm=torch.ones(head_dim, device=device) if norms else None,
                           k_norm=torch.ones(head_dim, device=device) if norms else None)


def main():
    layer = random_layer(bits=4, norms=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    vocabulary = 32000
    embedding = (torch.randn((vocabulary, 1024), generator=g, device="cuda")).to(torch.bfloat16)
    settings = {"temperature": 0.8, "top_p": 0.95, "min_p": 0.01}
    head = TokenHead(random_nbits(1024, vocabulary, g), layer.B,
                     **{n: torch.full((layer.B,), v, device="cuda") for n, v in settings.items()})
    tokens = torch.zeros((layer.B,), dtype=torch.int32, device="cuda")
    out = torch.empty((layer.B, 1024), dtype=torch.bfloat16, device="cuda")
    for step in range(200):
        x = embedding[tokens.long()]
        layer.step(x, out)
        tokens = head.step(torch.nn.functional.normalize((x + out).float(), dim=-1).mul_(32).to(torch.bfloat16),
                           torch.rand((layer.B,), generator=g, device="cuda"))
        if step % 50 == 49:
            print(f"step {step + 1}: cached {layer.length}, tokens {tokens.tolist()}, "
                  f"mean log-probability {head.logprobs.mean():.3f}")
    q.sync_status()


if __name__ == "__main__":
    main()
